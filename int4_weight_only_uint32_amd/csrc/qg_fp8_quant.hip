// Per-row, per-128-column e4m3 quantization of fp16/bf16 activations, plain or
// of the product silu(gate) * up, the input stage of the block-scaled fp8 GEMM.
//   scale = max |x| / 448,  code = e4m3(clamp(x / scale, -448, 448))
//
// Bound by memory: each value is read once and its code written once.  Sixteen
// lanes hold a block of 128, 8 values (one 16-byte word) each, so a wave's load is
// 1 KB without gaps.  One block per 16 lanes: more in flight per workgroup (R
// runs of 16 blocks) measured slower, 85 us for R = 1, 89 for 2 and 95 for 4 on 4096
// rows of a 2 x 17408 bf16 pair (360 MB), 2.3, 3.1 and 5.0 on 16 x 5120.  With the
// codes as below the pair takes 75 to 77 us, 4.7 TB/s, as a copy does.
//
// The code of x at scale sc is that of the correctly rounded quotient x / sc.
// The division is costly (ten instructions a value), so the code is first taken
// from y = x * inv, inv = 1 / sc correctly rounded, twice: of y a little
// smaller and a little larger, by more than y and the rounded quotient can
// differ.  Equal codes are the quotient's too (rounding is monotone); only where
// they are not, next to a border between two codes, is the division done.
//
// silu(gate) * up is formed in binary32 and is some steps off, which alone would
// move a few codes and most scales by a step.  The same two codes tell where a
// step could matter, and there the value is formed again in 64 bits; so is
// the block's largest value, for the scale.  Codes and scales are then those of
// the product in 64 bits.
#include "qg_device.h"
#include "qg_launch.h"

namespace qg {
namespace {

struct QuantShape {
    int K, KB;
    unsigned blocks;        // M * KB, below 2^28
    unsigned magic;         // blk / KB = blk * magic >> shift
    int shift;
};

template <bool BF16>
__device__ inline void widen8(const uint4v &a, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = BF16 ? bf2f((uint16_t)a[j]) : h2f((uint16_t)a[j]);
        x[2 * j + 1] = BF16 ? bf2f((uint16_t)(a[j] >> 16)) : h2f((uint16_t)(a[j] >> 16));
    }
}

// silu(g) in binary32 within 2^-22 of its size for g > -87; below, a value of
// less than SILU_SMALL (a NaN or infinity gives a NaN or an infinity).
constexpr float SILU_SMALL = 0x1p-100f;
__device__ inline float silu_near(float g)
{
    const float x = __builtin_fminf(__builtin_fmaxf(-g, -87.0f), 87.0f);
    return g * rcp_near(1.0f + exp_near(x));
}

__device__ inline double silu_64(float g, float u)
{
    return (double)g / (1.0 + exp(-(double)g)) * (double)u;
}

// Four e4m3 codes (nearest, ties to even; up to 464 gives 448, a NaN a NaN).
__device__ inline unsigned code4(float a, float b, float c, float d)
{
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

template <bool BF16, bool SWIGLU>
__global__ __launch_bounds__(256) void quantize_rows_fp8_kernel(
    const uint16_t *__restrict__ A, QuantShape q, uint8_t *__restrict__ Aq,
    float *__restrict__ a_scale)
{
    const int sub = threadIdx.x & 15;
    const unsigned blk = blockIdx.x * 16 + (threadIdx.x >> 4);
    if (blk >= q.blocks) return;       // all 16 lanes of a block
    const unsigned row = (unsigned)(((unsigned long long)blk * q.magic) >> q.shift);
    const int k = (int)(blk - row * q.KB) * 128 + sub * 8;
    const bool in = k < q.K;
    const size_t at = (size_t)row * q.K + k;
    uint4v g = {0u, 0u, 0u, 0u}, u = g;
    if (in) {
        const uint16_t *p = A + at + (SWIGLU ? (size_t)row * q.K : 0);
        g = __builtin_nontemporal_load(reinterpret_cast<const uint4v *>(p));
        if (SWIGLU) u = __builtin_nontemporal_load(reinterpret_cast<const uint4v *>(p + q.K));
    }
    float x[8], y[8];
    widen8<BF16>(g, x);
    if (SWIGLU) {
        widen8<BF16>(u, y);
        float least = __builtin_inff();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = silu_near(x[j]);
            least = __builtin_fminf(least, __builtin_fabsf(s));
            x[j] = s * y[j];
        }
        if (least < SILU_SMALL) {
            // A bf16 up value may raise a silu near or below binary32's least values
            // back to any size: those in 64 bits.
            float xg[8];
            widen8<BF16>(g, xg);
            unsigned redo = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                redo |= (xg[j] < -60.0f || (__builtin_fabsf(xg[j]) < 2 * SILU_SMALL && xg[j] != 0.0f) ? 1u : 0u) << j;
            while (redo) {
                const int at_j = __builtin_ctz(redo);
                float gj = 0.f, uj = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    gj = j == at_j ? xg[j] : gj;
                    uj = j == at_j ? y[j] : uj;
                }
                const float v = (float)silu_64(gj, uj);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = j == at_j ? v : x[j];
                redo &= redo - 1;
            }
        }
    }
    // magnitudes as bit patterns: ordered as the values are, NaN above infinity
    unsigned mx = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        mx = __builtin_elementwise_max(mx, __builtin_bit_cast(unsigned, x[j]) & 0x7fffffffu);
    // over the 16 lanes of a block, by rotations of a row of 16
#define QG_ROT_MAX(v, ctrl) \
    v = __builtin_elementwise_max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false))
#define QG_ROW_MAX(v) QG_ROT_MAX(v, 0x128); QG_ROT_MAX(v, 0x124); QG_ROT_MAX(v, 0x122); QG_ROT_MAX(v, 0x121)
    QG_ROW_MAX(mx);
    float sc;
    if (mx >= 0x7f800000u) {
        sc = __builtin_nanf("");
    } else if (SWIGLU) {
        // the values that may be the largest: those within 2^-19 of it; all where
        // binary32 holds them with fewer bits
        const float big = __builtin_bit_cast(float, mx), near = big < 0x1p-100f ? 0.f : big * (1.0f - 0x1p-19f);
        unsigned cand = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) cand |= (__builtin_fabsf(x[j]) >= near && mx ? 1u : 0u) << j;
        unsigned best = 0;
        while (cand) {       // (one lane of the 16, once, as a rule)
            float gj = 0.f, uj = 0.f, xg[8];
            widen8<BF16>(g, xg);
            const int at_j = __builtin_ctz(cand);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                gj = j == at_j ? xg[j] : gj;
                uj = j == at_j ? y[j] : uj;
            }
            const float s = (float)(__builtin_fabs(silu_64(gj, uj)) / 448.0);
            best = __builtin_elementwise_max(best, __builtin_bit_cast(unsigned, s));
            cand &= cand - 1;
        }
        mx = mx ? best : 0u;
        QG_ROW_MAX(mx);
        sc = __builtin_bit_cast(float, mx);
    } else {
        sc = __builtin_bit_cast(float, mx) / 448.0f;
    }
    if (sub == 0) a_scale[blk] = sc;
    if (!in) return;
    // y is off by 2 2^-24 (the inverse and the product), the rounded quotient by
    // 2^-24, silu by up to 2^-21
    constexpr float EPS = SWIGLU ? 0x1p-20f : 0x1p-21f;
    const float inv = sc > 0.0f ? 1.0f / sc : sc;        // 0 for a block of zeros, NaN for a NaN
    uint2v o, o2;
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = x[j] * inv;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        o[h] = code4(t[4 * h] * (1.f - EPS), t[4 * h + 1] * (1.f - EPS), t[4 * h + 2] * (1.f - EPS), t[4 * h + 3] * (1.f - EPS));
        o2[h] = code4(t[4 * h] * (1.f + EPS), t[4 * h + 1] * (1.f + EPS), t[4 * h + 2] * (1.f + EPS), t[4 * h + 3] * (1.f + EPS));
    }
    // (a scale so small that its inverse may overflow: every value)
    const bool small = sc < 0x1p-100f && sc > 0.0f;
    if (o.x != o2.x || o.y != o2.y || small) {
        float xg[8];
        if (SWIGLU) widen8<BF16>(g, xg);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned differ = (o[j / 4] ^ o2[j / 4]) >> (8 * (j & 3)) & 0xffu;
            if (differ || small) {
                const float v = SWIGLU ? (float)(silu_64(xg[j], y[j]) / (double)sc) : x[j] / sc;
                const unsigned c = code4(v > 448.f ? 448.f : v < -448.f ? -448.f : v, 0.f, 0.f, 0.f) & 0xffu;
                o[j / 4] = (o[j / 4] & ~(0xffu << (8 * (j & 3)))) | c << (8 * (j & 3));
            }
        }
    }
    // no scale, no sign either: -0 and what is too small for a scale are the byte 0 too
    if (sc == 0.0f) o = uint2v{0u, 0u};
    __builtin_nontemporal_store(o, reinterpret_cast<uint2v *>(Aq + at));
}
#undef QG_ROW_MAX
#undef QG_ROT_MAX

} // namespace

hipError_t launch_quantize_rows_fp8(const void *A, int dtype, int M, int K, bool swiglu,
                                    uint8_t *Aq, float *a_scale, hipStream_t st)
{
    QuantShape q;
    q.K = K;
    q.KB = (int)((K + 127ll) / 128);      // (K up to 2^31 - 16)
    q.blocks = (unsigned)M * (unsigned)q.KB;
    // blk < 2^28: magic = ceil(2^(29 + l) / KB) <= 2^30 with 2^l >= KB is off by less
    // than blk * KB / 2^(29 + l) < 1 part of a block
    int l = 0;
    while ((1ll << l) < q.KB) ++l;
    q.shift = 29 + l;
    q.magic = (unsigned)(((1ull << q.shift) + q.KB - 1) / q.KB);
    const dim3 block(256);
    const uint16_t *a = (const uint16_t *)A;
#define QG_QUANT8(BF, SW) \
    hipLaunchKernelGGL((quantize_rows_fp8_kernel<BF, SW>), dim3((q.blocks + 15) / 16), block, 0, st, a, q, Aq, a_scale)
    if (dtype == QG_DT_BF16) {
        if (swiglu) QG_QUANT8(true, true);
        else QG_QUANT8(true, false);
    } else {
        if (swiglu) QG_QUANT8(false, true);
        else QG_QUANT8(false, false);
    }
#undef QG_QUANT8
    return hipGetLastError();
}

} // namespace qg
