// Per-row, per-128-column e4m3 quantization of fp16/bf16 activations, plain or
// of the product silu(gate) * up, the input stage of the block-scaled fp8 GEMM.
//   scale = max |x| / 448,  code = e4m3(clamp(x / scale, -448, 448))
//
// Bound by memory: each value is read once and its code written once.  Sixteen
// lanes hold a block of 128, 8 values (one 16-byte word) each, so a wave's load is
// 1 KB without gaps.  One block per 16 lanes: more in flight per workgroup (R
// runs of 16 blocks) measured slower, 85 us for R = 1, 89 for 2 and 95 for 4 on 4096
// rows of a 2 x 17408 bf16 pair (360 MB), 2.3, 3.1 and 5.0 on 16 x 5120.
//
// The code of x at scale sc is that of the correctly rounded quotient x / sc.
// The division is costly (ten instructions a value: at 4096 rows of a
// 2 x 17408 pair the kernel took 97 us with it), so the code is first taken
// from y = x * inv, inv = 1 / sc correctly rounded: y is at most 2 steps of
// binary32 from x / sc (two roundings of relative size 2^-24), the rounded
// quotient half a step, so both are on the same side of every border between
// two codes unless y is within 3 steps of one.  Borders of normal codes have
// binary32's low 20 fraction bits equal to 0x80000.  Only next to them, below
// 2^-6 (the codes' subnormals) and for scales whose inverse could overflow is
// the division done.
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

// silu(g) * u in binary32, a few steps off.  Below -88 silu is 0 to 2e-37 |g|;
// infinities and NaN give a NaN or an infinity.
__device__ inline float silu_near(float g, float u)
{
    const float x = __builtin_fminf(__builtin_fmaxf(-g, -87.0f), 88.0f);
    const float s = rcp_near(1.0f + exp_near(x));
    return g * (g > -88.0f ? s : 0.0f) * u;
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
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = silu_near(x[j], y[j]);
    }
    // magnitudes as bit patterns: ordered as the values are, NaN above infinity
    unsigned mx = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        mx = __builtin_elementwise_max(mx, __builtin_bit_cast(unsigned, x[j]) & 0x7fffffffu);
    // over the 16 lanes of a block, by rotations of a row of 16
#define QG_DPP_MAX(ctrl) \
    mx = __builtin_elementwise_max(mx, (unsigned)__builtin_amdgcn_update_dpp(0, (int)mx, ctrl, 0xf, 0xf, false))
    QG_DPP_MAX(0x128);
    QG_DPP_MAX(0x124);
    QG_DPP_MAX(0x122);
    QG_DPP_MAX(0x121);
#undef QG_DPP_MAX
    float sc = __builtin_bit_cast(float, mx) / 448.0f;
    if (mx >= 0x7f800000u) sc = __builtin_nanf("");
    if (sub == 0) a_scale[blk] = sc;
    if (!in) return;
    const float inv = mx ? 1.0f / sc : 0.0f;
    bool redo = sc < 0x1p-100f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = x[j] * inv;
        const unsigned b = __builtin_bit_cast(unsigned, y[j]);
        redo |= ((b - 0x7fffdu) & 0xfffffu) <= 6u || __builtin_fabsf(y[j]) < 0x1p-6f;
    }
    if (redo && mx) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j] / sc;
    }
    uint2v o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 4 * h; j < 4 * h + 4; ++j)
            // (a NaN passes both comparisons)
            y[j] = y[j] > 448.f ? 448.f : y[j] < -448.f ? -448.f : y[j];
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], w, true);
        o[h] = (unsigned)w;
    }
    __builtin_nontemporal_store(o, reinterpret_cast<uint2v *>(Aq + at));
}

} // namespace

hipError_t launch_quantize_rows_fp8(const void *A, int dtype, int M, int K, bool swiglu,
                                    uint8_t *Aq, float *a_scale, hipStream_t st)
{
    QuantShape q;
    q.K = K;
    q.KB = (K + 127) / 128;
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
