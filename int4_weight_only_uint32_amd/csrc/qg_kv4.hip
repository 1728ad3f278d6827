// Rows of keys and values into the paged 4-bit cache (rotated and quantized on the
// way) and back out of it; the layout is qg_kv4.h's.
#include "qg_kv4.h"
#include "qg_launch.h"

namespace qg {
namespace {

constexpr int THREADS = 256;

template <bool BF16>
__device__ inline float to_f(uint16_t b) { return BF16 ? bf2f(b) : h2f(b); }
template <bool BF16>
__device__ inline uint16_t from_f(float f) { return BF16 ? f2bf(f) : f2h(f); }

typedef uint16_t ushort8v __attribute__((ext_vector_type(8)));

// Eight channels from d on of a row, rotated by the angles of position `at`.  Each
// product and each sum is rounded once (no fused multiply-add): the same bits whatever
// the compiler would contract, so a row's codes follow from the formula alone.
template <bool BF16>
__device__ inline void rotated8(const uint16_t *__restrict__ row, int d, int rot, bool inter,
                                const float *__restrict__ cos_sin, int at, int positions, float *x)
{
#pragma clang fp contract(off)
    const ushort8v own = *reinterpret_cast<const ushort8v *>(row + d);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f<BF16>(own[i]);
    if (d >= rot) return;
    const int half = rot / 2;
    if ((unsigned)at >= (unsigned)positions) {       // no angles for it
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
        return;
    }
    const float *const t = cos_sin + (size_t)at * rot;
    if (inter) {
        const float4v c = *reinterpret_cast<const float4v *>(t + d / 2);
        const float4v s = *reinterpret_cast<const float4v *>(t + half + d / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * c[i] - b * s[i];
            x[2 * i + 1] = b * c[i] + a * s[i];
        }
        return;
    }
    const bool first = d < half;
    const int e = first ? d : d - half;
    const ushort8v oth = *reinterpret_cast<const ushort8v *>(row + (first ? d + half : e));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = t[e + i], s = t[half + e + i], o = to_f<BF16>(oth[i]);
        x[i] = first ? x[i] * c - o * s : x[i] * c + o * s;
    }
}

struct AppendArgs {
    const uint16_t *k, *v, *q;
    long long ldk, ldv, ldq;       // elements from one token's row to the next
    int q_heads;
    const int32_t *positions;
    const float *cos_sin;
    int rot, max_pos;
    bool inter;
    uint16_t *q_out;
};

// One workgroup a 32-token block of one head's keys, or of its values, or of eight
// query heads.  A value word holds eight tokens, so the block's owner reads the words
// that it fills only in part; no other workgroup touches them.  Bound by memory (the
// rows in, the query rows out); a thread takes eight channels (16 bytes).
template <int D, bool BF16>
__global__ __launch_bounds__(THREADS) void kv4_append_kernel(Kv4Cache c, Kv4Batch s, AppendArgs a)
{
    constexpr int TPT = D / 8;                 // threads a token
    constexpr int STEP = THREADS / TPT;        // tokens at a time
    constexpr int QH = 8;                      // query heads of a workgroup
    __shared__ __attribute__((aligned(16))) uint8_t code[KV4_BLOCK][D];
    const int tid = threadIdx.x;
    int b, in, of;
    Run seq;
    if (!kv4_find(s, blockIdx.x, [](const Run &q) { return kv4_row_blocks(q); }, b, in, of, seq)) return;
    const int first = seq.len - seq.n;                      // index of the first new row
    const int t0 = ((first >> 5) + in) << 5;                // the block's first token
    const int lo = first > t0 ? first - t0 : 0;             // new rows: lo .. hi - 1 of the block
    const int hi = seq.len - t0 < KV4_BLOCK ? seq.len - t0 : KV4_BLOCK;
    const int y = blockIdx.y, d = tid % TPT * 8;

    if (y >= 2 * c.heads) {                                 // queries
        const int h0 = (y - 2 * c.heads) * QH;
        const int hs = a.q_heads - h0 < QH ? a.q_heads - h0 : QH;
        for (int i = tid / TPT; i < (hi - lo) * hs; i += STEP) {
            const int r = i / hs, h = h0 + i - r * hs, t = t0 + lo + r;
            const size_t row = (size_t)seq.row + (t - first);
            const int at = a.positions ? a.positions[row] : t;
            float x[8];
            rotated8<BF16>(a.q + row * a.ldq + (size_t)h * D, d, a.rot, a.inter, a.cos_sin, at, a.max_pos, x);
            ushort8v o;
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = from_f<BF16>(x[j]);
            *reinterpret_cast<ushort8v *>(a.q_out + (row * a.q_heads + h) * D + d) = o;
        }
        return;
    }

    const bool val = y >= c.heads;
    const int h = val ? y - c.heads : y;
    const int pg = kv4_page(c, s, b, t0);
    if (pg < 0) return;                                     // no place: nothing is stored
    const size_t head = (size_t)pg * c.heads + h;
    const int in_page = t0 & ((1 << c.shift) - 1);
    uint32_t *const words = (val ? c.v : c.k) + ((head << c.shift) + in_page) * (D / 8);
    uint32_t *const sz = (val ? c.v_sz : c.k_sz) + ((head * (c.D / c.g)) << c.shift) + in_page;

    for (int t = lo + tid / TPT; t < hi; t += STEP) {
        const size_t row = (size_t)seq.row + (t0 + t - first);
        float x[8];
        if (val)
            rotated8<BF16>(a.v + row * a.ldv + (size_t)h * D, d, 0, false, nullptr, 0, 0, x);
        else
            rotated8<BF16>(a.k + row * a.ldk + (size_t)h * D, d, a.rot, a.inter, a.cos_sin,
                           a.positions ? a.positions[row] : t0 + t, a.max_pos, x);
        float mn = x[0], mx = x[0];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mn = fminf(mn, x[j]);
            mx = fmaxf(mx, x[j]);
            bad |= x[j] != x[j];
        }
        // the threads of a group are neighbours: g / 8 = 4, 8 or 16 lanes
        for (int o = 1; o < c.g / 8; o <<= 1) {
            mn = fminf(mn, __shfl_xor(mn, o));
            mx = fmaxf(mx, __shfl_xor(mx, o));
            bad |= __shfl_xor((int)bad, o) != 0;
        }
        const uint16_t zb = f2h(mn);
        // past binary16 (or no number): the group says so, and so does every sum with it
        bad |= (zb & 0x7C00) == 0x7C00 || (f2h(mx) & 0x7C00) == 0x7C00;
        const uint16_t sb = bad ? 0x7E00 : f2h((mx - mn) / 15.0f);
        const float sc = h2f(sb), z = h2f(zb);
        uint64_t packed = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = sc > 0.0f ? rintf((x[j] - z) / sc) : 0.0f;
            v = v < 0.0f ? 0.0f : (v > 15.0f ? 15.0f : v);
            packed |= (uint64_t)(uint32_t)v << (8 * j);
        }
        *reinterpret_cast<uint64_t *>(&code[t][d]) = packed;
        if (d % c.g == 0) sz[((d / c.g) << c.shift) + t] = (uint32_t)sb | (uint32_t)(bad ? 0x7E00 : zb) << 16;
    }
    debug_stage_sync();
    __syncthreads();

    constexpr int WT = D / 8;                               // words a token
    if (!val) {
        for (int i = lo * WT + tid; i < hi * WT; i += THREADS) {
            const int t = i / WT, w = i % WT, q = w / (D / 32), j = w % (D / 32);
            const int base = 32 * (j >> 1) + 8 * q + 4 * (j & 1);
            const uint32_t l = *reinterpret_cast<const uint32_t *>(&code[t][base]);
            const uint32_t u = *reinterpret_cast<const uint32_t *>(&code[t][base + D / 2]);
            // byte 2b + a of l is nibble 4a + 2b, of u nibble 4a + 2b + 1
            const uint32_t m = l | u << 4;
            words[i] = (m & 0xFF) | (m & 0xFF0000) >> 8 | (m & 0xFF00) << 8 | (m & 0xFF000000);
        }
        return;
    }
    for (int i = tid; i < KV4_BLOCK * WT; i += THREADS) {
        const int j = i & 3, m = i >> 2 & 15, q = i >> 6 & 3, u = i >> 8;
        const int ch = 64 * u + 16 * j + m;
        uint32_t w = 0, mask = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int t = 16 * (n & 1) + 4 * q + 2 * (n >> 1 & 1) + (n >> 2);
            if (t >= lo && t < hi) {
                w |= (uint32_t)code[t][ch] << (4 * n);
                mask |= 15u << (4 * n);
            }
        }
        if (mask == 0) continue;
        words[i] = mask == 0xFFFFFFFFu ? w : (words[i] & ~mask) | w;
    }
}

// One workgroup a 32-token block of one head's keys or values: the block's words
// through LDS, eight channels a thread.  Bound by the 16-bit rows that it writes.
template <int D, int DT>
__global__ __launch_bounds__(THREADS) void kv4_read_kernel(Kv4Cache c, Kv4Batch s, void *k_out, void *v_out)
{
    constexpr int TPT = D / 8, STEP = THREADS / TPT, WT = D / 8;
    __shared__ uint32_t wl[KV4_BLOCK * WT];
    const int tid = threadIdx.x;
    int b, in, of;
    Run seq;
    if (!kv4_find(s, blockIdx.x, [](const Run &q) { return kv4_row_blocks(q); }, b, in, of, seq)) return;
    const int first = seq.len - seq.n;
    const int t0 = ((first >> 5) + in) << 5;
    const int lo = first > t0 ? first - t0 : 0;
    const int hi = seq.len - t0 < KV4_BLOCK ? seq.len - t0 : KV4_BLOCK;
    const bool val = (int)blockIdx.y >= c.heads;
    const int h = val ? blockIdx.y - c.heads : blockIdx.y;
    const int pg = kv4_page(c, s, b, t0);
    const size_t head = (size_t)(pg < 0 ? 0 : pg) * c.heads + h;
    const int in_page = pg < 0 ? 0 : t0 & ((1 << c.shift) - 1);
    const uint32_t *const words = (val ? c.v : c.k) + ((head << c.shift) + in_page) * WT;
    const uint32_t *const sz = (val ? c.v_sz : c.k_sz) + ((head * (c.D / c.g)) << c.shift) + in_page;
    for (int i = tid; i < KV4_BLOCK * WT; i += THREADS) wl[i] = words[i];
    debug_stage_sync();
    __syncthreads();
    const int d = tid % TPT * 8;
    for (int t = lo + tid / TPT; t < hi; t += STEP) {
        float x[8];
        const uint32_t p = sz[((d / c.g) << c.shift) + t];
        const float sc = h2f((uint16_t)p), z = h2f((uint16_t)(p >> 16));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            int at, nib;
            if (val) {
                nib = 4 * (t & 1) + 2 * (t >> 1 & 1) + (t >> 4);
                at = (((d >> 6) * 4 + (t >> 2 & 3)) * 16 + (d & 15) + j) * 4 + (d >> 4 & 3);
            } else {
                // channel 32 step + 8 q + j of the token
                const int step = d >> 5, q = d >> 3 & 3, up = step >= D / 64;
                nib = 4 * (j & 1) + 2 * (j >> 1 & 1) + up;
                at = t * WT + q * (D / 32) + 2 * (step - (up ? D / 64 : 0)) + (j >> 2);
            }
            x[j] = (float)(wl[at] >> (4 * nib) & 15) * sc + z;
            if (pg < 0) x[j] = 0.0f;
        }
        const size_t o = (((size_t)seq.row + (t0 + t - first)) * c.heads + h) * D + d;
        void *const out = val ? v_out : k_out;
        if (DT == QG_DT_F32) {
            float *const f = (float *)out + o;
            *reinterpret_cast<float4v *>(f) = float4v{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<float4v *>(f + 4) = float4v{x[4], x[5], x[6], x[7]};
        } else {
            ushort8v r;
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = from_f<DT == QG_DT_BF16>(x[j]);
            *reinterpret_cast<ushort8v *>((uint16_t *)out + o) = r;
        }
    }
}

} // namespace

long long kv4_blocks_bound(int T, int B) { return kv4_row_blocks_bound(T, B); }

hipError_t launch_kv4_append(const Kv4Cache &c, const Kv4Batch &s, const void *k, const void *v, const void *q,
                             long long ldk, long long ldv, long long ldq, int q_heads, int dtype,
                             const int32_t *positions, const float *cos_sin, int rot, int max_pos, bool inter,
                             void *q_out, hipStream_t st)
{
    const AppendArgs a = {(const uint16_t *)k, (const uint16_t *)v, (const uint16_t *)q, ldk, ldv, ldq, q_heads,
                          positions, cos_sin, rot, max_pos, inter, (uint16_t *)q_out};
    const dim3 grid((unsigned)kv4_row_blocks_bound(s.T, s.B), 2 * c.heads + (q ? (q_heads + 7) / 8 : 0));
#define QG_APPEND(D)                                                                                       \
    if (dtype == QG_DT_BF16)                                                                               \
        hipLaunchKernelGGL((kv4_append_kernel<D, true>), grid, dim3(THREADS), 0, st, c, s, a);             \
    else                                                                                                   \
        hipLaunchKernelGGL((kv4_append_kernel<D, false>), grid, dim3(THREADS), 0, st, c, s, a)
    switch (c.D) {
    case 64: QG_APPEND(64); break;
    case 128: QG_APPEND(128); break;
    case 256: QG_APPEND(256); break;
    default: return hipErrorInvalidValue;
    }
#undef QG_APPEND
    return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache &c, const Kv4Batch &s, int dtype, void *k_out, void *v_out, hipStream_t st)
{
    const dim3 grid((unsigned)kv4_row_blocks_bound(s.T, s.B), 2 * c.heads);
#define QG_READ(D)                                                                                         \
    if (dtype == QG_DT_F32)                                                                                \
        hipLaunchKernelGGL((kv4_read_kernel<D, QG_DT_F32>), grid, dim3(THREADS), 0, st, c, s, k_out, v_out);   \
    else if (dtype == QG_DT_BF16)                                                                          \
        hipLaunchKernelGGL((kv4_read_kernel<D, QG_DT_BF16>), grid, dim3(THREADS), 0, st, c, s, k_out, v_out);  \
    else                                                                                                   \
        hipLaunchKernelGGL((kv4_read_kernel<D, QG_DT_F16>), grid, dim3(THREADS), 0, st, c, s, k_out, v_out)
    switch (c.D) {
    case 64: QG_READ(64); break;
    case 128: QG_READ(128); break;
    case 256: QG_READ(256); break;
    default: return hipErrorInvalidValue;
    }
#undef QG_READ
    return hipGetLastError();
}

} // namespace qg
