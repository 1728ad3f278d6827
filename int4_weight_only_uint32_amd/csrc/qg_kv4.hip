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

// How a row is rotated (the same for all of a call): its first rot channels, channel i with
// channel i + rot / 2, or (PAIRS) with its neighbour; NONE: as it stands.
enum Turn { NONE, HALVES, PAIRS };

// Eight channels from d on of a row as they stand, with their partners.
struct Eight {
    ushort8v own, other;
};
template <Turn TURN>
__device__ inline Eight load8(const uint16_t *row, int d, int rot)
{
    Eight r;
    r.own = *reinterpret_cast<const ushort8v *>(row + d);
    if (TURN == HALVES) {
        const int half = rot / 2, e = d >= rot ? d : d < half ? d + half : d - half;
        r.other = *reinterpret_cast<const ushort8v *>(row + e);
    }
    return r;
}

// The cosines and sines of those channels at position `at` (of pairs: four of each), the sines
// negative where a channel is the first of its pair.  Without angles for the position none of
// them is a number, and so is no rotated channel.  Channels past rot get a cosine of 1 and
// a sine of -0: x * 1 + 0 * -0 is x, bit for bit.
struct Angles {
    float c[8], s[8];
    bool in;
};
template <Turn TURN>
__device__ inline Angles load_angles(const float *cos_sin, int d, int rot, int at, int positions)
{
    Angles r;
    if (TURN == NONE) return r;
    r.in = d < rot;
    const bool known = (unsigned)at < (unsigned)positions, first = TURN == HALVES && d < rot / 2;
    const float *const t = cos_sin + (size_t)(known ? at : 0) * rot;
    const int e = !r.in ? 0 : TURN == PAIRS ? d / 2 : first ? d : d - rot / 2;
#pragma unroll
    for (int i = 0; i < (TURN == PAIRS ? 4 : 8); i += 4) {
        const float4v c = *reinterpret_cast<const float4v *>(t + e + i);
        const float4v s = *reinterpret_cast<const float4v *>(t + rot / 2 + e + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r.c[i + j] = !r.in ? 1.0f : known ? c[j] : __builtin_nanf("");
            r.s[i + j] = !r.in ? -0.0f : first ? -s[j] : s[j];
        }
    }
    return r;
}

// The channels rotated.  Each product and each sum is rounded once (no fused
// multiply-add): the same bits whatever the compiler would contract, so a row's codes follow
// from the formula alone.
template <Turn TURN, bool BF16>
__device__ inline void rotate8(const Eight &r, const Angles &a, float *x)
{
#pragma clang fp contract(off)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f<BF16>(r.own[i]);
    if (TURN == PAIRS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = x[2 * i], v = x[2 * i + 1], p = a.in ? u : 0.0f, q = a.in ? v : -0.0f;
            x[2 * i] = u * a.c[i] + q * -a.s[i];
            x[2 * i + 1] = v * a.c[i] + p * a.s[i];
        }
    } else if (TURN == HALVES) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * a.c[i] + (a.in ? to_f<BF16>(r.other[i]) : 0.0f) * a.s[i];
    }
}

// 1 / d within two steps for d of 2^-24 .. 2^17: the hardware's reciprocal and a Newton step.
__device__ inline float rcp_wide(float d)
{
    const float y = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, y, 1.0f), y, y);
}

struct AppendArgs {
    const uint16_t *k, *v, *q;
    long long ldk, ldv, ldq;       // elements from one token's row to the next
    int q_heads;
    const int32_t *positions;
    const float *cos_sin;
    int rot, max_pos;
    uint16_t *q_out;
};

// One workgroup a 32-token block of one head's keys, or of its values, or of four
// query heads (these first: they are the most).  A value word holds eight tokens, so the
// block's owner reads the words that it fills only in part; no other workgroup touches them.
// Bound by memory (the rows in, the query rows out); a thread takes eight channels (16
// bytes).  Rows of three prompts of up to 2731 tokens, 8 heads of 128 and 40 query heads: 43 us,
// one token 5.6.
constexpr int QUERY_HEADS = 4;
template <int D, Turn TURN, bool BF16>
__global__ __launch_bounds__(THREADS, D < 256 ? 6 : 4) void kv4_append_kernel(Kv4Cache c, Kv4Batch s, AppendArgs a)
{
    constexpr int TPT = D / 8;                 // threads a token
    constexpr int STEP = THREADS / TPT;        // tokens at a time
    constexpr int QH = QUERY_HEADS;
    __shared__ __attribute__((aligned(16))) uint8_t code[KV4_BLOCK][D];
    const int tid = threadIdx.x;
    int b, in, of;
    Run seq;
    if (!kv4_find(s, blockIdx.x, [](const Run &q) { return kv4_row_blocks(q); }, b, in, of, seq)) return;
    const int first = seq.len - seq.n;                      // index of the first new row
    const int t0 = ((first >> 5) + in) << 5;                // the block's first token
    const int lo = first > t0 ? first - t0 : 0;             // new rows: lo .. hi - 1 of the block
    const int hi = seq.len - t0 < KV4_BLOCK ? seq.len - t0 : KV4_BLOCK;
    const int groups = (a.q_heads + QH - 1) / QH, y = (int)blockIdx.y - groups, d = tid % TPT * 8;

    if (y < 0) {
        // queries: a thread keeps its channels of a token through the heads, all of them in flight
        const int h0 = (int)blockIdx.y * QH;
        const int hs = a.q_heads - h0 < QH ? a.q_heads - h0 : QH;
        for (int t = lo + tid / TPT; t < hi; t += STEP) {
            const size_t row = (size_t)seq.row + (t0 + t - first);
            const int at = a.positions ? a.positions[row] : t0 + t;
            const Angles an = load_angles<TURN>(a.cos_sin, d, a.rot, at, a.max_pos);
            const uint16_t *const q = a.q + row * a.ldq + (size_t)h0 * D;
            Eight r[QH];
#pragma unroll
            for (int h = 0; h < QH; ++h) r[h] = load8<TURN>(q + (h < hs ? h : 0) * D, d, a.rot);
#pragma unroll
            for (int h = 0; h < QH; ++h) {
                float x[8];
                rotate8<TURN, BF16>(r[h], an, x);
                ushort8v o;
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = from_f<BF16>(x[j]);
                if (h < hs) *reinterpret_cast<ushort8v *>(a.q_out + (row * a.q_heads + h0 + h) * D + d) = o;
            }
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

    // every token's loads first
    constexpr int PASSES = KV4_BLOCK / STEP;
    Eight raw[PASSES];
    Angles an[PASSES];
    const uint16_t *const src = (val ? a.v : a.k) + (size_t)h * D;
    const long long ld = val ? a.ldv : a.ldk;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        int t = tid / TPT + i * STEP;
        t = t < lo ? lo : t < hi ? t : hi - 1;
        const size_t row = (size_t)seq.row + (t0 + t - first);
        if (val) {
            raw[i] = load8<NONE>(src + row * ld, d, 0);
        } else {
            raw[i] = load8<TURN>(src + row * ld, d, a.rot);
            an[i] = load_angles<TURN>(a.cos_sin, d, a.rot, TURN != NONE && a.positions ? a.positions[row] : t0 + t, a.max_pos);
        }
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int t = tid / TPT + i * STEP;
        float x[8];
        if (val)
            rotate8<NONE, BF16>(raw[i], an[i], x);
        else
            rotate8<TURN, BF16>(raw[i], an[i], x);
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
        // (x - z) / s to the nearest whole number: by the reciprocal, whose product is within 2^-17
        // of a quotient up to 16 (16 times two steps, 2^-22, and a rounding, 2^-24), and by the
        // division where that lies within 2^-16 of the middle of two
        const float rs = sc > 0.0f ? rcp_wide(sc) : 0.0f;
        float q[8], near = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = (x[j] - z) * rs;
            q[j] = rintf(y);
            near = fmaxf(near, __builtin_fabsf(y - q[j]));
        }
        if (near > 0.5f - 0x1p-16f)
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = rintf((x[j] - z) / sc);
        uint2v packed = {0, 0};                            // (clamped to 0 .. 15; no number: 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fminf(fmaxf(q[j], 0.0f), 15.0f);
            packed[j >> 2] = __builtin_amdgcn_cvt_pk_u8_f32(v, j & 3, packed[j >> 2]);
        }
        *reinterpret_cast<uint2v *>(&code[t][d]) = packed;
        if (t >= lo && t < hi && d % c.g == 0) sz[((d / c.g) << c.shift) + t] = (uint32_t)sb | (uint32_t)(bad ? 0x7E00 : zb) << 16;
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
    const bool whole = lo == 0 && hi == KV4_BLOCK;
    for (int i = tid; i < KV4_BLOCK * WT; i += THREADS) {
        const int j = i & 3, m = i >> 2 & 15, q = i >> 6 & 3, u = i >> 8;
        const int ch = 64 * u + 16 * j + m;
        uint32_t w = 0, mask = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int t = 16 * (n & 1) + 4 * q + 2 * (n >> 1 & 1) + (n >> 2);
            w |= (uint32_t)code[t][ch] << (4 * n);
            mask |= !whole && t >= lo && t < hi ? 15u << (4 * n) : 0u;
        }
        if (whole)
            words[i] = w;
        else if (mask != 0)
            words[i] = (words[i] & ~mask) | (w & mask);
    }
}

// A wave a 32-token block of HPW heads' keys or values, four waves side by side; all of a wave's
// loads are in flight together.  A lane gives out eight channels of a token (16 bytes) at a
// time: of keys from two words that stand together, of values, where they are the same
// nibble of eight words, through LDS.  Bound by the 16-bit rows that it writes: 8 x 16000 tokens
// of 8 heads of 128 in 98 us (5.1 TB/s with the codes, a copy's rate), 777 tokens in 5.
template <int D, int DT, int HPW>
__global__ __launch_bounds__(THREADS) void kv4_read_kernel(Kv4Cache c, Kv4Batch s, void *k_out, void *v_out)
{
    constexpr int TPT = D / 8, STEP = 64 / TPT, WT = D / 8, ITEMS = KV4_BLOCK / STEP, LOADS = D / 64;
    __shared__ __attribute__((aligned(16))) uint32_t lds[4][KV4_BLOCK * WT];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int b, in, of;
    Run seq;
    if (!kv4_find(s, blockIdx.x, [](const Run &q) { return kv4_row_blocks(q); }, b, in, of, seq)) return;
    const int first = seq.len - seq.n;
    const int t0 = ((first >> 5) + in) << 5;
    const int lo = first > t0 ? first - t0 : 0;
    const int hi = seq.len - t0 < KV4_BLOCK ? seq.len - t0 : KV4_BLOCK;
    const int groups = gridDim.y / 2;
    const bool val = (int)blockIdx.y >= groups;
    const int h0 = (blockIdx.y - (val ? groups : 0)) * 4 * HPW + w;
    if (h0 >= c.heads) return;                              // (no barrier below)
    const int pg = kv4_page(c, s, b, t0);
    const int in_page = pg < 0 ? 0 : t0 & ((1 << c.shift) - 1);
    const int d = lane % TPT * 8, tl = lane / TPT;
    const uint32_t *const codes = val ? c.v : c.k, *const scales = val ? c.v_sz : c.k_sz;
    void *const out = val ? v_out : k_out;

    uint4v vw[HPW][LOADS];
    uint2v kw[HPW][ITEMS];
    uint32_t sz[HPW][ITEMS];
    const int step = d >> 5, up = step >= D / 64;           // of keys: the k-step and its half of the nibbles
    const int kat = (d >> 3 & 3) * (D / 32) + 2 * (step - (up ? D / 64 : 0));
#pragma unroll
    for (int i = 0; i < HPW; ++i) {
        const int h = h0 + 4 * i < c.heads ? h0 + 4 * i : h0;
        const size_t head = (size_t)(pg < 0 ? 0 : pg) * c.heads + h;
        const uint32_t *const words = codes + ((head << c.shift) + in_page) * WT;
        if (val) {
#pragma unroll
            for (int u = 0; u < LOADS; ++u) vw[i][u] = *reinterpret_cast<const uint4v *>(words + u * 256 + lane * 4);
        } else {
#pragma unroll
            for (int it = 0; it < ITEMS; ++it) kw[i][it] = *reinterpret_cast<const uint2v *>(words + (it * STEP + tl) * WT + kat);
        }
#pragma unroll
        for (int it = 0; it < ITEMS; ++it)
            sz[i][it] = scales[((head * (c.D / c.g) + d / c.g) << c.shift) + in_page + it * STEP + tl];
    }
#pragma unroll
    for (int i = 0; i < HPW; ++i) {
        const int h = h0 + 4 * i;
        if (h >= c.heads) break;
        if (val) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // (the head before has been read)
#pragma unroll
            for (int u = 0; u < LOADS; ++u) *reinterpret_cast<uint4v *>(&lds[w][u * 256 + lane * 4]) = vw[i][u];
            debug_stage_sync();
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
#pragma unroll
        for (int it = 0; it < ITEMS; ++it) {
            const int t = it * STEP + tl;
            const float sc = h2f((uint16_t)sz[i][it]), z = h2f((uint16_t)(sz[i][it] >> 16));
            float x[8];
            if (val) {
                const int sh = 4 * (4 * (t & 1) + 2 * (t >> 1 & 1) + (t >> 4));
                const uint32_t *const p = &lds[w][(((d >> 6) * 4 + (t >> 2 & 3)) * 16 + (d & 15)) * 4 + (d >> 4 & 3)];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = (float)(p[4 * j] >> sh & 15) * sc + z;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int sh = 4 * (4 * (j & 1) + 2 * (j >> 1 & 1));
                    x[j] = (float)((j < 4 ? kw[i][it].x : kw[i][it].y) >> (up ? sh + 4 : sh) & 15) * sc + z;
                }
            }
            if (pg < 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            if (t < lo || t >= hi) continue;
            const size_t o = (((size_t)seq.row + (t0 + t - first)) * c.heads + h) * D + d;
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
}

} // namespace

long long kv4_blocks_bound(int T, int B) { return kv4_row_blocks_bound(T, B); }

hipError_t launch_kv4_append(const Kv4Cache &c, const Kv4Batch &s, const void *k, const void *v, const void *q,
                             long long ldk, long long ldv, long long ldq, int q_heads, int dtype,
                             const int32_t *positions, const float *cos_sin, int rot, int max_pos, bool inter,
                             void *q_out, hipStream_t st)
{
    const AppendArgs a = {(const uint16_t *)k, (const uint16_t *)v, (const uint16_t *)q, ldk, ldv, ldq,
                          q ? q_heads : 0, positions, cos_sin, rot, max_pos, (uint16_t *)q_out};
    const dim3 grid((unsigned)kv4_row_blocks_bound(s.T, s.B), 2 * c.heads + (a.q_heads + QUERY_HEADS - 1) / QUERY_HEADS);
#define QG_APPEND2(DIM, TURN)                                                                          \
    if (dtype == QG_DT_BF16)                                                                           \
        hipLaunchKernelGGL((kv4_append_kernel<DIM, TURN, true>), grid, dim3(THREADS), 0, st, c, s, a); \
    else                                                                                               \
        hipLaunchKernelGGL((kv4_append_kernel<DIM, TURN, false>), grid, dim3(THREADS), 0, st, c, s, a)
#define QG_APPEND(DIM)                \
    if (rot == 0) {                   \
        QG_APPEND2(DIM, NONE);        \
    } else if (inter) {               \
        QG_APPEND2(DIM, PAIRS);       \
    } else {                          \
        QG_APPEND2(DIM, HALVES);      \
    }
    switch (c.D) {
    case 64: QG_APPEND(64); break;
    case 128: QG_APPEND(128); break;
    case 256: QG_APPEND(256); break;
    default: return hipErrorInvalidValue;
    }
#undef QG_APPEND
#undef QG_APPEND2
    return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache &c, const Kv4Batch &s, int dtype, void *k_out, void *v_out, hipStream_t st)
{
    // two heads a wave where one a wave fills the CUs several times over
    const long long blocks = kv4_row_blocks_bound(s.T, s.B);
    const int hpw = blocks * 2 * ((c.heads + 3) / 4) > 4096 ? 2 : 1;
    const dim3 grid((unsigned)blocks, 2 * ((c.heads + 4 * hpw - 1) / (4 * hpw)));
#define QG_READ2(DIM, DTYPE)                                                                                   \
    if (hpw == 2)                                                                                              \
        hipLaunchKernelGGL((kv4_read_kernel<DIM, DTYPE, 2>), grid, dim3(THREADS), 0, st, c, s, k_out, v_out);  \
    else                                                                                                       \
        hipLaunchKernelGGL((kv4_read_kernel<DIM, DTYPE, 1>), grid, dim3(THREADS), 0, st, c, s, k_out, v_out)
#define QG_READ(DIM)                        \
    if (dtype == QG_DT_F32) {               \
        QG_READ2(DIM, QG_DT_F32);           \
    } else if (dtype == QG_DT_BF16) {       \
        QG_READ2(DIM, QG_DT_BF16);          \
    } else {                                \
        QG_READ2(DIM, QG_DT_F16);           \
    }
    switch (c.D) {
    case 64: QG_READ(64); break;
    case 128: QG_READ(128); break;
    case 256: QG_READ(256); break;
    default: return hipErrorInvalidValue;
    }
#undef QG_READ
#undef QG_READ2
    return hipGetLastError();
}

} // namespace qg
