// Low-rank adapters of many requests beside a shared projection:
//   Y[t] += scaling[a] * (X[t] . A[a]^T) . B[a]^T
// for the tokens t of adapter a, which stand together in the sorted order of
// moe_sort_rows.  Two launches (three where adapters have many rows), on the 16-bit MFMA: the narrow product H = X . A^T,
// split along K into partial sums (32 bits, in the workspace, added in a fixed order), and
// the wide one, which reads and writes Y.  Bound by reading X, the adapters in use and Y,
// and by writing Y.
//
// H is not rounded to 16 bits between the two: a row's values (64 of them at a time), scaled
// by a power of two, go into the second product as the sum of two 16-bit values (22 bits for
// fp16, 16 for bf16), which costs a second MFMA where memory is the bound.
#include <type_traits>

#include "qg_launch.h"
#include "qg_ragged.h"

namespace qg {
namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));

template <bool BF16>
__device__ inline float4v mfma16(uint4v a, uint4v b, float4v c)
{
    if (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}
template <bool BF16>
__device__ inline float to_f(uint16_t b) { return BF16 ? bf2f(b) : h2f(b); }
template <bool BF16>
__device__ inline uint16_t from_f(float f) { return BF16 ? f2bf(f) : f2h(f); }

struct LoraArgs {
    const uint16_t *x, *a, *b;
    const float *scaling;
    const int32_t *off, *rows, *slots;
    uint16_t *y;
    float *part;                   // [splits][T][R]: the sorted rows of H, a part of K each
    uint16_t *h;                   // [T][2][Rp]: upper and lower parts of their sums
    int32_t *ex;                   // [T][chunks]: the power of two of 64 of a row's values
    int L, T, K, N, R, splits, Rp, chunks;
};

constexpr int CHUNK = 64;          // columns of H with one power of two

template <int BM>
__device__ inline bool find_rows(const LoraArgs &p, int x, int &e, int &m0, int &end)
{
    int in, of;
    Run r;
    if (!find_item(p.L, x, [&](int i) { return i < p.L ? run_of(p.off, p.T, i) : Run{0, 0, 0}; },
                   [](const Run &q) { return (q.n + BM - 1) / BM; }, e, in, of, r))
        return false;
    m0 = r.row + in * BM;
    end = r.row + r.n;
    return true;
}

// H for 16 MT rows and 16 RT columns (of a chunk of 64) of one adapter, over one of `splits`
// parts of K: four waves take quarters of the part and add up through LDS.  Rows without
// a token (and columns past R) are computed from row 0 and come to nothing.  Bound by reading X
// and A, few rows by the latency of one step after another: 64 rows of K = 5120, 32 adapters of
// rank 16 5.0 us, 4093 rows, 8 of rank 64 22.6 (42 MB of X).
template <int MT, int RT, bool BF16>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs p)
{
    constexpr int BM = 16 * MT;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, kq = lane >> 4;
    const int split = blockIdx.y, r0 = blockIdx.z * CHUNK;
    int e, m0, end;
    if (!find_rows<BM>(p, blockIdx.x, e, m0, end)) return;
    const uint16_t *xr[MT], *ar[RT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + 16 * i + col;
        int t = p.rows[m < end ? m : m0];
        t = (unsigned)t < (unsigned)p.T ? t : 0;
        xr[i] = p.x + (size_t)t * p.K + 8 * kq;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = r0 + 16 * i + col;
        ar[i] = p.a + ((size_t)e * p.R + (r < p.R ? r : 0)) * p.K + 8 * kq;
    }
    float4v acc[MT][RT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = float4v{0, 0, 0, 0};
    const int whole = p.K / 64, steps = (p.K + 63) / 64, parts = p.splits * 4;
    const int per = (steps + parts - 1) / parts, s0 = (split * 4 + w) * per;
    const int s1 = s0 + per < whole ? s0 + per : whole;
    struct Step {
        uint4v x[2][MT], a[2][RT];
    };
    auto load = [&](int s, Step &v) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < MT; ++i) v.x[u][i] = *reinterpret_cast<const uint4v *>(xr[i] + 64 * s + 32 * u);
#pragma unroll
            for (int j = 0; j < RT; ++j) v.a[u][j] = *reinterpret_cast<const uint4v *>(ar[j] + 64 * s + 32 * u);
        }
    };
    auto add = [&](const Step &v) {
        debug_stage_sync();
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[i][j] = mfma16<BF16>(v.a[u][j], v.x[u][i], acc[i][j]);
    };
    // a step's loads are in flight while the one before is added
    if (s0 < s1) {
        Step v[2];
        load(s0, v[0]);
        for (int s = s0; s < s1; s += 2) {
            load(s + 1 < s1 ? s + 1 : s, v[1]);
            __builtin_amdgcn_sched_barrier(0);             // (not later, where they would take fewer registers)
            add(v[0]);
            if (s + 1 >= s1) break;
            load(s + 2 < s1 ? s + 2 : s + 1, v[0]);
            __builtin_amdgcn_sched_barrier(0);
            add(v[1]);
        }
    }
    if (whole < steps && s0 <= whole && whole < s0 + per) {
        // (K is a multiple of eight: a lane's eight k are all there or none)
        Step v;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = 64 * whole + 32 * u;
            const bool in = k + 8 * kq < p.K;
            const uint4v zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MT; ++i) v.x[u][i] = in ? *reinterpret_cast<const uint4v *>(xr[i] + k) : zero;
#pragma unroll
            for (int j = 0; j < RT; ++j) v.a[u][j] = in ? *reinterpret_cast<const uint4v *>(ar[j] + k) : zero;
        }
        add(v);
    }
    __shared__ float4v sum[4][MT * RT][64];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) sum[w][i * RT + j][lane] = acc[i][j];
    debug_stage_sync();
    __syncthreads();
    for (int i = w; i < MT * RT; i += 4) {
        const float4v v = sum[0][i][lane] + sum[1][i][lane] + (sum[2][i][lane] + sum[3][i][lane]);
        const int m = m0 + 16 * (i / RT) + col, r = r0 + 16 * (i % RT) + 4 * kq;
        if (m < end && r < p.R)
            *reinterpret_cast<float4v *>(p.part + ((size_t)split * p.T + m) * p.R + r) = v;
    }
}

// Eight values of H's sorted row m from column r on, summed over the parts of K in order.
__device__ inline void row8(const LoraArgs &p, int m, int r, float by, float *v)
{
    float4v a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (r < p.R) {
        const float *h = p.part + (size_t)m * p.R + r;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s, h += (size_t)p.T * p.R) {
            a += *reinterpret_cast<const float4v *>(h);
            b += *reinterpret_cast<const float4v *>(h + 4);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        v[u] = a[u] * by;
        v[4 + u] = b[u] * by;
    }
}

// Eight values as two of 16 bits each, after scaling by 2^-ex.
template <bool BF16>
__device__ inline void two_parts(const float *v, int ex, uint4v &hi, uint4v &lo)
{
    hi = lo = uint4v{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const float f = ldexpf(v[u], -ex);
        const uint16_t hb = from_f<BF16>(f);
        const uint16_t lb = __builtin_fabsf(f) < __builtin_inff() ? from_f<BF16>(f - to_f<BF16>(hb)) : 0;
        hi[u >> 1] |= (unsigned)hb << (16 * (u & 1));
        lo[u >> 1] |= (unsigned)lb << (16 * (u & 1));
    }
}

// The power of two above `big` (0 for a row of zeros or no numbers).
__device__ inline int power_of(float big)
{
    int ex = 0;
    if (big > 0.0f && big < __builtin_inff()) (void)frexpf(big, &ex);
    return ex;
}

__device__ inline float largest(const float *v)
{
    float big = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) big = fmaxf(big, __builtin_fabsf(v[u]));
    return big;
}

// For the tall kernel, whose workgroups would each sum the same rows: H's rows summed and
// split once (4093 rows of rank 64: 4.9 us).  A row's adapter is the one
// whose range holds it; eight threads a chunk of 64.
template <bool BF16>
__global__ __launch_bounds__(256) void lora_split_kernel(LoraArgs p)
{
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int part = id & 7;
    const long long q = id >> 3;
    const int m = (int)(q / p.chunks), ch = (int)(q - (long long)m * p.chunks);
    if (m >= p.T) return;
    // the last adapter whose range begins at or before m
    int lo_e = 0, hi_e = p.L;
    while (hi_e - lo_e > 1) {
        const int mid = (lo_e + hi_e) >> 1;
        if (p.off[mid] <= m) lo_e = mid; else hi_e = mid;
    }
    const float by = p.scaling ? p.scaling[lo_e] : 1.0f;
    const int r = CHUNK * ch + 8 * part;
    float v[8];
    row8(p, m, r, by, v);
    float big = largest(v);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) big = fmaxf(big, __shfl_xor(big, o));
    const int ex = power_of(big);
    uint4v hi, lo;
    two_parts<BF16>(v, ex, hi, lo);
    if (r < p.Rp) {
        uint16_t *const h = p.h + (size_t)m * 2 * p.Rp + r;
        *reinterpret_cast<uint4v *>(h) = hi;
        *reinterpret_cast<uint4v *>(h + p.Rp) = lo;
    }
    if (part == 0) p.ex[(size_t)m * p.chunks + ch] = ex;
}

// A lane's token of a row tile, -1 without one.  slots[t] is the one row of token t: a
// token that stands in two rows is taken in that one only, so no two waves write it.
__device__ inline int token_of(const LoraArgs &p, int m, int end)
{
    const int t = m < end ? p.rows[m] : -1;
    return (unsigned)t < (unsigned)p.T && p.slots[t] == m ? t : -1;
}

// In both wide kernels the adapter's rows are the MFMA's rows, tile j holding columns
// 32 (j / 2) + 8 (row / 4) + 4 (j % 2) + row % 4 of 64, so that a lane ends with twice eight
// consecutive columns of one token: 16 bytes, and 64 with its neighbours.
__device__ inline int column_of(int j, int row) { return 32 * (j >> 1) + 8 * (row >> 2) + 4 * (j & 1) + (row & 3); }

// A token's eight values with the adapter's part added.
template <bool BF16>
__device__ inline uint4v added(uint4v old, float4v a, float4v b)
{
    uint4v now = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        const float o = to_f<BF16>((uint16_t)(old[v >> 1] >> (16 * (v & 1))));
        now[v >> 1] |= (unsigned)from_f<BF16>(o + (v < 4 ? a[v & 3] : b[v & 3])) << (16 * (v & 1));
    }
    return now;
}

// Few rows an adapter: 16 rows, 64 columns a wave, four waves side by side, `strips` times
// after one another.  Loads stand outside of branches, at clamped places (what they bring
// there is not stored), so that all of a strip's are in flight together.  Bound by Y, read and
// written: 64 rows of 32 adapters, N = 17408 10.3 us, one row of 5120 5.9 (latency).
template <bool BF16>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs p, int strips, int ranges)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, kq = lane >> 4;
    int e, m0, end;
    if (!find_rows<16>(p, blockIdx.x / ranges, e, m0, end)) return;
    const int range = blockIdx.x % ranges;
    const int m = m0 + col, tok = token_of(p, m, end), mc = m < end ? m : m0;
    uint16_t *const yr = p.y + (size_t)(tok >= 0 ? tok : 0) * p.N;
    const uint16_t *const be = p.b + (size_t)e * p.N * p.R;
    const float by = p.scaling ? p.scaling[e] : 1.0f;
    // a chunk of the row of H as operands, and its power of two over the lane groups
    uint4v hi[2], lo[2];
    int ex;
    auto chunk = [&](int ch) {
        float v[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s) row8(p, mc, CHUNK * ch + 32 * s + 8 * kq, by, v[s]);
        float big = fmaxf(largest(v[0]), largest(v[1]));
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        ex = power_of(big);
#pragma unroll
        for (int s = 0; s < 2; ++s) two_parts<BF16>(v[s], ex, hi[s], lo[s]);
    };
    uint4v old[2], bv[4];
    auto load_y = [&](int nb) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int c = nb + 32 * u + 8 * kq;
            old[u] = *reinterpret_cast<const uint4v *>(yr + (c < p.N ? c : p.N - 8));
        }
    };
    auto load_b = [&](int nb, int r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = nb + column_of(j, col);
            bv[j] = *reinterpret_cast<const uint4v *>(be + (size_t)(c < p.N ? c : p.N - 1) * p.R + (r < p.R ? r : 0));
        }
    };
    const int first = (range * strips * 4 + w) * 64;
    if (first >= p.N) return;
    load_y(first);
    load_b(first, 8 * kq);
    chunk(0);
    for (int n = 0; n < strips; ++n) {
        const int nb = first + 256 * n;
        if (nb >= p.N) return;
        if (n > 0) {
            load_y(nb);
            load_b(nb, 8 * kq);
        }
        float4v all[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
        for (int ch = 0; ch < p.chunks; ++ch) {
            float4v acc[4] = {{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
            if (p.chunks > 1) chunk(ch);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int r = CHUNK * ch + 32 * s + 8 * kq;
                if (s == 1 && CHUNK * ch + 32 >= p.R) break;
                if (s + ch > 0) load_b(nb, r);
                debug_stage_sync();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (r >= p.R) bv[j] = uint4v{0, 0, 0, 0};   // (zeros meet zeros, not what stands there)
                    acc[j] = mfma16<BF16>(bv[j], hi[s], acc[j]);
                    acc[j] = mfma16<BF16>(bv[j], lo[s], acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) all[j][v] += ldexpf(acc[j][v], ex);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int c = nb + 32 * u + 8 * kq;
            const uint4v now = added<BF16>(old[u], all[2 * u], all[2 * u + 1]);
            if (tok >= 0 && c < p.N) *reinterpret_cast<uint4v *>(yr + c) = now;
        }
    }
}

// Many rows an adapter: 128 rows a workgroup, 32 a wave, which hold H's operands for good, and
// all four waves the same 64 columns at a time, their part of B (one run of memory) brought
// to LDS once for all of them, one strip ahead.  Workgroups go to the eight XCDs in turn and
// the column range is the fastest index: with eight ranges or more a range of B is read
// into one XCD's L2.  Bound by Y, read and written: 4093 rows of N = 17408, rank 64 82 us (3.5 TB/s).
template <int ST, bool BF16>
__global__ __launch_bounds__(256, 2) void lora_expand_tall_kernel(LoraArgs p, int strips, int ranges)
{
    constexpr int MT = 2, BM = 64 * MT, CH = (ST + 1) / 2;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, kq = lane >> 4;
    int e, m0, end;
    if (!find_rows<BM>(p, blockIdx.x / ranges, e, m0, end)) return;
    const int range = blockIdx.x % ranges;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][64 * 32 * ST * 2];
    // strip n's 8 R chunks of 16 bytes, R / 8 loads of 64 lanes; a chunk's place in a line of eight is
    // turned by its line's number, so that the operands' reads of 16 rows spread over the banks
    const int loads = p.R / 8;
    const size_t most = (size_t)p.N * p.R / 8 - 1;         // B[e]'s last chunk
    const uint16_t *const be = p.b + (size_t)e * p.N * p.R;
    auto turn = [](int line) { return ((line >> 3) * 4 + (line & 3)) & 7; };
    auto load_b = [&](int nb, int to) {
        for (int i = w; i < loads; i += 4) {
            const int line = 8 * i + (lane >> 3);
            size_t chunk = (size_t)nb * p.R / 8 + 8 * line + ((lane & 7) ^ turn(line));
            chunk = chunk < most ? chunk : most;
            lds_load16<0>(reinterpret_cast<const uint32_t *>(be + chunk * 8), lds[to] + i * 1024);
        }
    };
    const int nb0 = range * strips * 64;
    int count = nb0 < p.N ? (p.N - nb0 + 63) / 64 : 0;
    count = count < strips ? count : strips;
    if (count == 0) return;
    load_b(nb0, 0);

    int tok[MT];
    uint16_t *yr[MT];
    uint4v hi[MT][ST], lo[MT][ST];
    int ex[MT][CH];
    bool full = true;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + 32 * w + 16 * i + col, mc = m < end ? m : m0;
        tok[i] = token_of(p, m, end);
        full &= tok[i] >= 0;
        yr[i] = p.y + (size_t)(tok[i] >= 0 ? tok[i] : 0) * p.N;
        const uint16_t *const hr = p.h + (size_t)mc * 2 * p.Rp + 8 * kq;
#pragma unroll
        for (int s = 0; s < ST; ++s) {
            const bool in = 32 * s < p.Rp;
            hi[i][s] = *reinterpret_cast<const uint4v *>(hr + (in ? 32 * s : 0));
            lo[i][s] = *reinterpret_cast<const uint4v *>(hr + p.Rp + (in ? 32 * s : 0));
            if (!in) hi[i][s] = lo[i][s] = uint4v{0, 0, 0, 0};
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) ex[i][c] = p.ex[(size_t)mc * p.chunks + (c < p.chunks ? c : 0)];
    }
    full = __all(full);

    // A strip's values of Y are asked for one strip ahead too.  Where all of a wave's values are
    // stored (FULL), the stores of a strip need not be waited for with the next one's loads.
    constexpr int STORES = 2 * MT;
    struct Rows {
        uint4v y[MT][2];
    };
    auto load_y = [&](int nb, Rows &v) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = nb + 32 * u + 8 * kq;
                v.y[i][u] = *reinterpret_cast<const uint4v *>(yr[i] + (c < p.N ? c : p.N - 8));
            }
    };
    auto strip = [&](int n, const Rows &cur, Rows &next, auto is_full) {
        constexpr bool FULL = decltype(is_full)::value;
        const int nb = nb0 + 64 * n;
        // this strip's part of B has landed, for every wave, and the other buffer is done with
        if (FULL && n > 0)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(STORES) : "memory");
        else
            __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load_y(n + 1 < count ? nb + 64 : nb, next);
        if (n + 1 < count) load_b(nb + 64, (n + 1) & 1);
        debug_stage_sync();
        __builtin_amdgcn_sched_barrier(0);
        float4v all[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) all[i][j] = float4v{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float4v acc[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = float4v{0, 0, 0, 0};
#pragma unroll
            for (int s = 2 * c; s < 2 * c + 2 && s < ST; ++s) {
                const int r = 32 * s + 8 * kq;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int chunk = (column_of(j, col) * p.R + (r < p.R ? r : 0)) / 8, line = chunk >> 3;
                    uint4v bv = *reinterpret_cast<const uint4v *>(lds[n & 1] + line * 128 + ((chunk & 7) ^ turn(line)) * 16);
                    if (r >= p.R) bv = uint4v{0, 0, 0, 0};      // (zeros meet zeros, not what stands there)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        acc[i][j] = mfma16<BF16>(bv, hi[i][s], acc[i][j]);
                        acc[i][j] = mfma16<BF16>(bv, lo[i][s], acc[i][j]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) all[i][j][v] += ldexpf(acc[i][j][v], ex[i][c]);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = nb + 32 * u + 8 * kq;
                const uint4v now = added<BF16>(cur.y[i][u], all[i][2 * u], all[i][2 * u + 1]);
                if (FULL || (tok[i] >= 0 && c < p.N)) *reinterpret_cast<uint4v *>(yr[i] + c) = now;
            }
    };
    // (each wave passes `count` barriers, whichever loop it is in)
    Rows y[2];
    load_y(nb0, y[0]);
    const int whole = full ? (p.N - nb0) / 64 : 0, lead = whole < count ? whole : count;
    int n = 0;
    for (; n + 1 < lead; n += 2) {
        strip(n, y[0], y[1], std::true_type{});
        strip(n + 1, y[1], y[0], std::true_type{});
    }
    for (; n < count; ++n) {
        strip(n, y[0], y[1], std::false_type{});
        y[0] = y[1];
    }
}

} // namespace

LoraPlan lora_plan(int T, int L, int K, int N, int R)
{
    LoraPlan p;
    const long long some = T < L ? T : L;                  // adapters with a part of a tile
    // narrow product: 64 rows a tile where the adapters have 16, by the mean; K in parts that
    // give each CU a workgroup (4093 tokens, 71 tiles at K = 5120, both products: 3 parts 104 us,
    // 2 parts 109, 4 parts, a round and a bit, 112), each wave at least four 64-k steps
    p.narrow_rows = T > 16 * (long long)L ? 64 : 16;
    p.narrow = T / p.narrow_rows + some;
    const int rz = (R + CHUNK - 1) / CHUNK, steps = (K + 63) / 64;
    const long long tiles = p.narrow * rz, most = (steps + 15) / 16;
    long long s = tiles <= 128 ? 256 / tiles : tiles <= 256 ? 2 : 1;
    s = s > most ? most : s;
    p.splits = s < 1 ? 1 : s > 8 ? 8 : (int)s;
    p.tall = T > 32 * (long long)L && R <= 128;            // (by the mean)
    p.tiles = T / (p.tall ? 128 : 16) + some;
    // column ranges: about 1536 workgroups of the tall kernel (4093 tokens: 104 us; 1024: 111, 2048:
    // 106), 1024 of the other (64 tokens: 14.3 us; 768: 15.5, 1536: 16.8), in eights where
    // there are that many
    const long long wide = p.tall ? (N + 63) / 64 : (N + 255) / 256;
    long long n = ((p.tall ? 1536 : 1024) + p.tiles - 1) / p.tiles;
    n = n > wide ? wide : n;
    if (n > 8) n &= ~7ll;
    p.strips = (int)((wide + n - 1) / n);
    p.ranges = (int)((wide + p.strips - 1) / p.strips);
    if (p.ranges > 8) p.ranges = (p.ranges + 7) & ~7;
    const size_t Rp = (R + 31) / 32 * 32;
    p.bytes = (size_t)T * R * p.splits * sizeof(float);
    if (p.tall) p.bytes += (size_t)T * (2 * Rp * sizeof(uint16_t) + rz * sizeof(int32_t));
    return p;
}

hipError_t launch_lora(const LoraPlan &pl, const void *x, const void *a, const void *b, const float *scaling,
                       const int32_t *off, const int32_t *rows, const int32_t *slots, int L, int T, int K, int N, int R,
                       int dtype, void *y, void *ws, hipStream_t st)
{
    const int Rp = (R + 31) / 32 * 32, chunks = (R + CHUNK - 1) / CHUNK;
    float *const part = (float *)ws;
    uint16_t *const h = (uint16_t *)(part + (size_t)T * R * pl.splits);    // (16-byte aligned: R is a multiple of 8)
    const LoraArgs p = {(const uint16_t *)x, (const uint16_t *)a, (const uint16_t *)b, scaling, off, rows, slots,
                        (uint16_t *)y, part, h, (int32_t *)(h + (size_t)T * 2 * Rp), L, T, K, N, R, pl.splits, Rp, chunks};
    const bool bf = dtype == QG_DT_BF16;
    const dim3 narrow((unsigned)pl.narrow, pl.splits, chunks), grid((unsigned)(pl.tiles * pl.ranges));
#define QG_SHRINK(MT, RT)                                                                               \
    if (bf)                                                                                             \
        hipLaunchKernelGGL((lora_shrink_kernel<MT, RT, true>), narrow, dim3(256), 0, st, p);            \
    else                                                                                                \
        hipLaunchKernelGGL((lora_shrink_kernel<MT, RT, false>), narrow, dim3(256), 0, st, p)
    if (pl.narrow_rows == 16) {
        if (R <= 16) {
            QG_SHRINK(1, 1);
        } else if (R <= 32) {
            QG_SHRINK(1, 2);
        } else {
            QG_SHRINK(1, 4);
        }
    } else {
        if (R <= 16) {
            QG_SHRINK(4, 1);
        } else if (R <= 32) {
            QG_SHRINK(4, 2);
        } else {
            QG_SHRINK(4, 4);
        }
    }
#undef QG_SHRINK
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (pl.tall) {
        const dim3 g((unsigned)(((long long)T * chunks * 8 + 255) / 256));
        if (bf)
            hipLaunchKernelGGL((lora_split_kernel<true>), g, dim3(256), 0, st, p);
        else
            hipLaunchKernelGGL((lora_split_kernel<false>), g, dim3(256), 0, st, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
#define QG_TALL(ST)                                                                                     \
    if (bf)                                                                                             \
        hipLaunchKernelGGL((lora_expand_tall_kernel<ST, true>), grid, dim3(256), 0, st, p, pl.strips, pl.ranges);  \
    else                                                                                                \
        hipLaunchKernelGGL((lora_expand_tall_kernel<ST, false>), grid, dim3(256), 0, st, p, pl.strips, pl.ranges)
    if (!pl.tall) {
        if (bf)
            hipLaunchKernelGGL((lora_expand_kernel<true>), grid, dim3(256), 0, st, p, pl.strips, pl.ranges);
        else
            hipLaunchKernelGGL((lora_expand_kernel<false>), grid, dim3(256), 0, st, p, pl.strips, pl.ranges);
    } else if (R <= 32) {
        QG_TALL(1);
    } else if (R <= 64) {
        QG_TALL(2);
    } else {
        QG_TALL(4);
    }
#undef QG_TALL
    return hipGetLastError();
}

} // namespace qg
