// Per-row, per-128-column e4m3 quantization of fp16/bf16 activations, plain or
// of the product silu(gate) * up, the input stage of the block-scaled fp8 GEMM.
//   scale = max |x| / 448,  code = e4m3(clamp(x / scale, -448, 448))
// Eight lanes hold one block: 16 values each.
#include "qg_device.h"
#include "qg_launch.h"

namespace qg {
namespace {

template <bool BF16>
__device__ inline void load16(const uint16_t *p, float (&x)[16])
{
    const uint4v a = *reinterpret_cast<const uint4v *>(p), b = *reinterpret_cast<const uint4v *>(p + 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const unsigned w = j < 4 ? a[j] : b[j - 4];
        x[2 * j] = BF16 ? bf2f((uint16_t)w) : h2f((uint16_t)w);
        x[2 * j + 1] = BF16 ? bf2f((uint16_t)(w >> 16)) : h2f((uint16_t)(w >> 16));
    }
}

template <bool BF16, bool SWIGLU>
__global__ __launch_bounds__(256) void quantize_rows_fp8_kernel(
    const uint16_t *__restrict__ A, int M, int K, int KB, uint8_t *__restrict__ Aq,
    float *__restrict__ a_scale)
{
    const size_t blk = ((size_t)blockIdx.x * 256 + threadIdx.x) >> 3;
    if (blk >= (size_t)M * KB) return;     // the eight lanes of a block leave together
    const int row = (int)(blk / KB), b = (int)(blk % KB);
    const int k = b * 128 + (threadIdx.x & 7) * 16;
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.f;
    if (k < K) {
        const uint16_t *p = A + (size_t)row * (SWIGLU ? 2 * (size_t)K : (size_t)K) + k;
        load16<BF16>(p, x);
        if (SWIGLU) {
            float u[16];
            load16<BF16>(p + K, u);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = x[j] / (1.0f + expf(-x[j])) * u[j];
        }
    }
    // magnitudes as bit patterns: ordered as the values are, NaN above infinity
    unsigned mx = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        mx = __builtin_elementwise_max(mx, __builtin_bit_cast(unsigned, x[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = __builtin_elementwise_max(mx, (unsigned)__shfl_xor((int)mx, o));
    float sc = __builtin_bit_cast(float, mx) / 448.0f;
    if (mx >= 0x7f800000u) sc = __builtin_nanf("");
    if ((threadIdx.x & 7) == 0) a_scale[blk] = sc;
    if (k >= K) return;
    uint4v q;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = mx ? x[4 * h + j] / sc : 0.f;
            // (a NaN passes both comparisons)
            y[j] = y[j] > 448.f ? 448.f : y[j] < -448.f ? -448.f : y[j];
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
        q[h] = (unsigned)w;
    }
    *reinterpret_cast<uint4v *>(Aq + (size_t)row * K + k) = q;
}

} // namespace

hipError_t launch_quantize_rows_fp8(const void *A, int dtype, int M, int K, bool swiglu,
                                    uint8_t *Aq, float *a_scale, hipStream_t st)
{
    const int KB = (K + 127) / 128;
    const size_t wgs = ((size_t)M * KB + 31) / 32;
    const dim3 grid((unsigned)wgs), block(256);
    const uint16_t *a = (const uint16_t *)A;
#define QG_QUANT8(BF, SW) \
    hipLaunchKernelGGL((quantize_rows_fp8_kernel<BF, SW>), grid, block, 0, st, a, M, K, KB, Aq, a_scale)
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
