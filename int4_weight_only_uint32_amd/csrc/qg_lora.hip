// Low-rank adapters of many requests beside a shared projection:
//   Y[t] += scaling[a] * (X[t] . A[a]^T) . B[a]^T
// for the tokens t of adapter a, which stand together in the sorted order of
// moe_sort_rows.  Two launches: the narrow product H = X . A^T, split along K into
// partial sums (32 bits, in the workspace, added in a fixed order), and the wide one, which
// reads and writes Y.  Both on the 16-bit MFMA; bound by reading X, the adapters
// in use and Y, and by writing Y.
//
// H is not rounded to 16 bits between the two: its row, scaled by a power of two, goes
// into the second product as the sum of two 16-bit values (22 bits for fp16, 16 for
// bf16), which costs a second MFMA where memory is the bound.
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
    float *h;                      // [splits][T][R]
    int L, T, K, N, R, splits;
};

// The token of sorted row m, -1 if it has none.  slots[t] is the one row of token t: a
// token that stands in two rows is taken in that one only, so no two waves write it.
__device__ inline int token_of(const LoraArgs &p, int m, int end)
{
    if (m >= end) return -1;
    const int t = p.rows[m];
    return (unsigned)t < (unsigned)p.T && p.slots[t] == m ? t : -1;
}

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

// H[m, r] for 16 MT rows and 16 RT columns of one adapter, over one of `splits` parts of K;
// the four waves take quarters of the part and add up through LDS.  A lane's 16
// consecutive k feed two MFMAs, so four lanes read a 128-byte line of a row.
template <int MT, int RT, bool BF16>
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs p)
{
    constexpr int BM = 16 * MT;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, kq = lane >> 4;
    const int split = blockIdx.y, r0 = blockIdx.z * 16 * RT;
    int e, m0, end;
    if (!find_rows<BM>(p, blockIdx.x, e, m0, end)) return;
    const uint16_t *xr[MT], *ar[RT];
    bool live[MT], has[RT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int t = token_of(p, m0 + 16 * i + col, end);
        live[i] = t >= 0;
        xr[i] = p.x + (size_t)(live[i] ? t : 0) * p.K;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = r0 + 16 * i + col;
        has[i] = r < p.R;
        ar[i] = p.a + ((size_t)e * p.R + (has[i] ? r : 0)) * p.K;
    }
    float4v acc[MT][RT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = float4v{0, 0, 0, 0};
    const int steps = (p.K + 63) / 64, parts = p.splits * 4;
    const int per = (steps + parts - 1) / parts, s0 = (split * 4 + w) * per;
    const int s1 = s0 + per < steps ? s0 + per : steps;
    const uint4v zero = {0, 0, 0, 0};
    for (int s = s0; s < s1; ++s) {
        const int k = 64 * s + 16 * kq;
        uint4v xv[MT][2], av[RT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const bool in = k + 8 * u < p.K;
#pragma unroll
            for (int i = 0; i < MT; ++i)
                xv[i][u] = in && live[i] ? *reinterpret_cast<const uint4v *>(xr[i] + k + 8 * u) : zero;
#pragma unroll
            for (int j = 0; j < RT; ++j)
                av[j][u] = in && has[j] ? *reinterpret_cast<const uint4v *>(ar[j] + k + 8 * u) : zero;
        }
        debug_stage_sync();
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[i][j] = mfma16<BF16>(av[j][u], xv[i][u], acc[i][j]);
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
            *reinterpret_cast<float4v *>(p.h + ((size_t)split * p.T + m) * p.R + r) = v;
    }
}

// Y for 16 MT rows and 64 columns a wave (four waves side by side, `strips` of them
// after one another).  The adapter's rows are the MFMA's rows, tile i holding columns
// 16 (row / 4) + 4 i + row % 4, so that a lane ends with 16 consecutive columns of
// one token: 32 bytes, and 128 with its neighbours.
template <int MT, bool BF16>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs p, int strips)
{
    constexpr int BM = 16 * MT;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = lane & 15, kq = lane >> 4;
    int e, m0, end;
    if (!find_rows<BM>(p, blockIdx.x, e, m0, end)) return;
    int tok[MT], m[MT], ex[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        m[i] = m0 + 16 * i + col;
        tok[i] = token_of(p, m[i], end);
    }
    const float by = p.scaling ? p.scaling[e] : 1.0f;
    // eight values of H's row m[i] from column r on
    auto row8 = [&](int i, int r, float *v) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = 0.0f;
        if (tok[i] < 0 || r >= p.R) return;
        for (int s = 0; s < p.splits; ++s) {
            const float *const h = p.h + ((size_t)s * p.T + m[i]) * p.R + r;
            const float4v a = *reinterpret_cast<const float4v *>(h), b = *reinterpret_cast<const float4v *>(h + 4);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u] += a[u];
                v[4 + u] += b[u];
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= by;
    };
    const int steps = (p.R + 31) / 32;
    // each row's power of two: its largest value below 1
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        float big = 0.0f;
        for (int s = 0; s < steps; ++s) {
            float v[8];
            row8(i, 32 * s + 8 * kq, v);
#pragma unroll
            for (int u = 0; u < 8; ++u) big = fmaxf(big, __builtin_fabsf(v[u]));
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        ex[i] = 0;
        if (big > 0.0f && big < __builtin_inff()) (void)frexpf(big, &ex[i]);
    }
    const uint4v zero = {0, 0, 0, 0};
    for (int n = 0; n < strips; ++n) {
        const int nb = ((blockIdx.y * strips + n) * 4 + w) * 64;
        if (nb >= p.N) return;
        float4v acc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = float4v{0, 0, 0, 0};
        for (int s = 0; s < steps; ++s) {
            const int r = 32 * s + 8 * kq;
            uint4v bv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = nb + 16 * (col >> 2) + 4 * j + (col & 3);
                bv[j] = c < p.N && r < p.R
                            ? *reinterpret_cast<const uint4v *>(p.b + ((size_t)e * p.N + c) * p.R + r) : zero;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float v[8];
                row8(i, r, v);
                uint4v hi = zero, lo = zero;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float f = ldexpf(v[u], -ex[i]);
                    const uint16_t hb = from_f<BF16>(f);
                    const float rest = f - to_f<BF16>(hb);
                    const uint16_t lb = __builtin_fabsf(f) < __builtin_inff() ? from_f<BF16>(rest) : 0;
                    hi[u >> 1] |= (unsigned)hb << (16 * (u & 1));
                    lo[u >> 1] |= (unsigned)lb << (16 * (u & 1));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = mfma16<BF16>(bv[j], hi, acc[i][j]);
                    acc[i][j] = mfma16<BF16>(bv[j], lo, acc[i][j]);
                }
            }
        }
        debug_stage_sync();
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (tok[i] < 0) continue;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = nb + 16 * kq + 8 * u;
                if (c >= p.N) continue;
                uint4v *const y = reinterpret_cast<uint4v *>(p.y + (size_t)tok[i] * p.N + c);
                uint4v old = *y, now = zero;
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    const float o = to_f<BF16>((uint16_t)(old[v >> 1] >> (16 * (v & 1))));
                    const float d = ldexpf(acc[i][2 * u + (v >> 2)][v & 3], ex[i]);
                    now[v >> 1] |= (unsigned)from_f<BF16>(o + d) << (16 * (v & 1));
                }
                *y = now;
            }
        }
    }
}

} // namespace

LoraPlan lora_plan(int T, int L, int K, int N, int R)
{
    LoraPlan p;
    p.mt = T > 16 * (long long)L ? 4 : 1;
    const int bm = 16 * p.mt;
    p.tiles = T / bm + (long long)(T < L ? T : L);
    const int rz = (R + 63) / 64, steps = (K + 63) / 64;
    long long s = (512 + p.tiles * rz - 1) / (p.tiles * rz);
    const long long most = (steps + 3) / 4;
    s = s > most ? most : s;
    s = s > 32 ? 32 : s;
    p.splits = s < 1 ? 1 : (int)s;
    const long long wide = (N + 255) / 256;
    p.strips = 1;
    while (p.strips < 8 && p.tiles * ((wide + p.strips - 1) / p.strips) > 2048) p.strips *= 2;
    p.bytes = (size_t)p.splits * T * R * sizeof(float);
    return p;
}

hipError_t launch_lora(const LoraPlan &pl, const void *x, const void *a, const void *b, const float *scaling,
                       const int32_t *off, const int32_t *rows, const int32_t *slots, int L, int T, int K, int N, int R,
                       int dtype, void *y, void *ws, hipStream_t st)
{
    const LoraArgs p = {(const uint16_t *)x, (const uint16_t *)a, (const uint16_t *)b, scaling, off, rows, slots,
                        (uint16_t *)y, (float *)ws, L, T, K, N, R, pl.splits};
    const bool bf = dtype == QG_DT_BF16;
#define QG_SHRINK(MT, RT)                                                                                           \
    {                                                                                                               \
        const dim3 grid((unsigned)pl.tiles, pl.splits, (R + 16 * RT - 1) / (16 * RT));                              \
        if (bf)                                                                                                     \
            hipLaunchKernelGGL((lora_shrink_kernel<MT, RT, true>), grid, dim3(256), 0, st, p);                      \
        else                                                                                                        \
            hipLaunchKernelGGL((lora_shrink_kernel<MT, RT, false>), grid, dim3(256), 0, st, p);                     \
    }
    if (pl.mt == 1) {
        if (R <= 16) QG_SHRINK(1, 1)
        else if (R <= 32) QG_SHRINK(1, 2)
        else QG_SHRINK(1, 4)
    } else {
        if (R <= 16) QG_SHRINK(4, 1)
        else if (R <= 32) QG_SHRINK(4, 2)
        else QG_SHRINK(4, 4)
    }
#undef QG_SHRINK
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int wide = (N + 255) / 256;
    const dim3 grid((unsigned)pl.tiles, (wide + pl.strips - 1) / pl.strips);
    if (pl.mt == 1) {
        if (bf)
            hipLaunchKernelGGL((lora_expand_kernel<1, true>), grid, dim3(256), 0, st, p, pl.strips);
        else
            hipLaunchKernelGGL((lora_expand_kernel<1, false>), grid, dim3(256), 0, st, p, pl.strips);
    } else {
        if (bf)
            hipLaunchKernelGGL((lora_expand_kernel<4, true>), grid, dim3(256), 0, st, p, pl.strips);
        else
            hipLaunchKernelGGL((lora_expand_kernel<4, false>), grid, dim3(256), 0, st, p, pl.strips);
    }
    return hipGetLastError();
}

} // namespace qg
