// Block-scaled fp8 GEMM, C = sum over 128-k blocks of a_scale * w_scale *
// (A . W^T), dense or grouped by expert, on the e4m3 MFMA whose k extent (128)
// is one scale block: each MFMA starts from zero and its result is one
// block's exact-scale partial product, folded into the fp32 accumulator with
// one FMA per value.
//
// The operands are swapped (W rows are the MFMA's rows, A rows its columns), so
// a lane's four results are four consecutive n of one row m: they share one
// activation scale, and store as one 8-byte word.
#include <cstdio>

#include "qg_device.h"
#include "qg_launch.h"

namespace qg {
namespace {

constexpr int KB8 = 128;   // k extent of a scale block, bytes of a tile row

// Rows of expert blocks.  The grid holds an upper bound on the number of
// BM-row blocks over all experts; block rb of the list is found by a scan over
// the offsets (64 experts a step, every wave for itself).
struct RowBlock {
    int e, m0, m1;      // expert, first row, end of the expert's rows; e < 0: none
};

__device__ inline RowBlock find_rows(const int32_t *__restrict__ offsets, int E, int M, int BM,
                                     int rb)
{
    if (!offsets) return RowBlock{rb * BM < M ? 0 : -1, rb * BM, M};
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int r0 = 0, r1 = 0;
        if (e0 + lane < E) {
            r0 = offsets[e0 + lane];
            r1 = offsets[e0 + lane + 1];
            r0 = r0 < 0 ? 0 : (r0 > M ? M : r0);
            r1 = r1 < r0 ? r0 : (r1 > M ? M : r1);
        }
        const int nb = (r1 - r0 + BM - 1) / BM;
        int sum = nb;      // inclusive scan
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned long long hit = __ballot(base + sum > rb);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int first = base + __shfl(sum - nb, l);
            return RowBlock{e0 + l, __shfl(r0, l) + (rb - first) * BM, __shfl(r1, l)};
        }
        base += __shfl(sum, 63);
    }
    return RowBlock{-1, 0, 0};
}

template <bool BF16>
__device__ inline uint16_t out16(float f) { return BF16 ? f2bf(f) : f2h(f); }

// ---- tiled kernel ----
// BM x BN tile per workgroup of WM x WN waves; each wave MT x NT 16 x 16
// tiles.  A 128-k step of both operands (rows of 128 bytes) is loaded straight
// to LDS, double-buffered, one barrier a step.  In LDS, 16-byte chunk c of row r
// stands at position c ^ (r % 8), so that the 16 rows a wave reads at once
// spread over the banks.
template <int BM, int BN, int WM, int WN, bool BF16>
__global__ __launch_bounds__(64 * WM * WN) void fp8_tiled_kernel(
    const uint8_t *__restrict__ Aall, const float *__restrict__ a_scale,
    const int32_t *__restrict__ a_rows, int M_a, const uint8_t *__restrict__ Wall,
    const float *__restrict__ Sall, const int32_t *__restrict__ offsets, int E, int M, int N,
    int K, int KB, int NB, uint16_t *__restrict__ C)
{
    constexpr int NW = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
    constexpr int LA = BM / 8 / NW, LW = BN / 8 / NW;    // 1 KB loads per wave and step
    static_assert(LA * NW * 8 == BM && LW * NW * 8 == BN, "whole loads per wave");
    static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0, "a wave's columns share one weight scale");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int STAGE = (BM + BN) * KB8;

    const int nbn = (N + BN - 1) / BN;
    const int rb = blockIdx.x / nbn, n0 = (blockIdx.x % nbn) * BN;
    const RowBlock blk = find_rows(offsets, E, M, BM, rb);
    if (blk.e < 0) return;      // uniform over the workgroup, before any barrier
    const int e = __builtin_amdgcn_readfirstlane(blk.e);
    const int m0 = __builtin_amdgcn_readfirstlane(blk.m0);
    const int m1 = __builtin_amdgcn_readfirstlane(blk.m1);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // every lane's source chunk within a row, and its rows' byte offsets; rows
    // past the end read the last row (never stored)
    const int chunk = (lane & 7) ^ (lane >> 3);
    const int rows_n = N - n0 < BN ? N - n0 : BN;
    const uint8_t *W = Wall + ((size_t)e * N + n0) * K;
    const __amdgpu_buffer_rsrc_t w_rs = buffer_rsrc(W, (size_t)rows_n * K);
    const __amdgpu_buffer_rsrc_t a_rs =
        a_rows ? buffer_rsrc(Aall, (size_t)M_a * K) : buffer_rsrc(Aall + (size_t)m0 * K, (size_t)(m1 - m0) * K);
    unsigned a_off[LA], w_off[LW];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        int r = (wave * LA + i) * 8 + (lane >> 3);
        r = m0 + r < m1 ? r : m1 - 1 - m0;
        if (a_rows) {
            r = a_rows[m0 + r];
            r = (unsigned)r < (unsigned)M_a ? r : 0;
        }
        a_off[i] = (unsigned)r * (unsigned)K + chunk * 16;
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        int r = (wave * LW + i) * 8 + (lane >> 3);
        r = r < rows_n ? r : rows_n - 1;
        w_off[i] = (unsigned)r * (unsigned)K + chunk * 16;
    }
    auto load = [&](int kt, int st) {
        // past the end of K (last step of a K that is no multiple of 128) an
        // offset beyond every range makes the load give zeros
        const bool in = kt * KB8 + chunk * 16 < K;
        uint8_t *base = lds + st * STAGE;
        // (plain variables of a fixed type: a target builtin given an argument
        // whose type depends on a template parameter loses the kernel's host
        // launch stub)
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const unsigned off = in ? a_off[i] + kt * KB8 : 0xFFFFFFF0u;
            uint8_t *dst = base + (wave * LA + i) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rs, (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            const unsigned off = in ? w_off[i] + kt * KB8 : 0xFFFFFFF0u;
            uint8_t *dst = base + BM * KB8 + (wave * LW + i) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rs, (__attribute__((address_space(3))) void *)dst, 16, off, 0, 0, 0);
        }
    };

    // scales: a lane's row of each m-tile, the wave's weight block
    const float *srow[MT];
    bool bad[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        int r = m0 + (wm * MT + t) * 16 + (lane & 15);
        r = r < m1 ? r : m1 - 1;
        bad[t] = false;
        if (a_rows) {
            r = a_rows[r];
            bad[t] = (unsigned)r >= (unsigned)M_a;
            r = bad[t] ? 0 : r;
        }
        srow[t] = a_scale + (size_t)r * KB;
    }
    int nb = (n0 + wn * NT * 16) / 128;
    nb = nb < NB ? nb : NB - 1;
    const float *sw = Sall + ((size_t)e * NB + nb) * KB;

    float4v acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};

    // operand position of this lane in a 16-row tile: chunks q and q ^ 4 of
    // lane group q = lane / 16
    const int o0 = (lane & 15) * KB8 + (((lane >> 4) ^ (lane & 7)) * 16);
    float sa[MT], sb = sw[0];      // the step's scales, loaded one step ahead
#pragma unroll
    for (int t = 0; t < MT; ++t) sa[t] = srow[t][0];
    load(0, 0);
    for (int kt = 0; kt < KB; ++kt) {
        // this step's tiles have landed, and every wave has read the last step's
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
        float s[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) s[t] = sa[t] * sb;
        if (kt + 1 < KB) {
            sb = sw[kt + 1];
#pragma unroll
            for (int t = 0; t < MT; ++t) sa[t] = srow[t][kt + 1];
            load(kt + 1, (kt + 1) & 1);
        }
        const uint8_t *At = lds + (kt & 1) * STAGE + wm * MT * 16 * KB8;
        const uint8_t *Wt = lds + (kt & 1) * STAGE + (BM + wn * NT * 16) * KB8;
        auto operand = [&](const uint8_t *p) {
            const int4v lo = *reinterpret_cast<const int4v *>(p + o0);
            const int4v hi = *reinterpret_cast<const int4v *>(p + (o0 ^ 64));
            return int8v{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        };
        int8v a[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) a[i] = operand(At + i * 16 * KB8);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int8v w = operand(Wt + j * 16 * KB8);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float4v p = mfma_fp8(w, a[i], float4v{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s[i], acc[i][j][r]);
            }
        }
    }

    const bool wide = N % 4 == 0 && ((uintptr_t)C & 7) == 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = m0 + (wm * MT + i) * 16 + (lane & 15);
        if (m >= m1) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = n0 + (wn * NT + j) * 16 + 4 * (lane >> 4);
            uint16_t h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = bad[i] ? 0 : out16<BF16>(acc[i][j][r]);
            uint16_t *c = C + (size_t)m * N + n;
            if (wide) {
                if (n < N)
                    *reinterpret_cast<uint2v *>(c) = uint2v{h[0] | (unsigned)h[1] << 16, h[2] | (unsigned)h[3] << 16};
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n + r < N) c[r] = h[r];
            }
        }
    }
}

struct Fp8Args {
    const uint8_t *A;
    const float *a_scale;
    const int32_t *a_rows;
    int M_a;
    const uint8_t *W;
    const float *w_scale;
    const int32_t *offsets;
    int E, M, N, K, KB, NB;
    uint16_t *C;
};

// Upper bound on the BM-row blocks of M rows in E experts: every non-empty
// expert may end in a partial block.
long long row_blocks(const Fp8Args &a, int BM)
{
    if (!a.offsets) return (a.M + BM - 1) / BM;
    return (long long)a.M / BM + (a.E < a.M ? a.E : a.M);
}

template <int BM, int BN, int WM, int WN, bool BF16>
hipError_t tiled(const Fp8Args &a, hipStream_t st)
{
    const auto kern = fp8_tiled_kernel<BM, BN, WM, WN, BF16>;
    constexpr int bytes = 2 * (BM + BN) * KB8;
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    const long long wgs = row_blocks(a, BM) * ((a.N + BN - 1) / BN);
    hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(64 * WM * WN), bytes, st, a.A, a.a_scale, a.a_rows,
                       a.M_a, a.W, a.w_scale, a.offsets, a.E, a.M, a.N, a.K, a.KB, a.NB, a.C);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch(const Fp8Args &a, hipStream_t st)
{
    return tiled<64, 128, 2, 2, BF16>(a, st);
}

} // namespace

hipError_t launch_fp8(const uint8_t *A, const float *a_scale, const int32_t *a_rows, int M_a,
                      const uint8_t *W, const float *w_scale, const int32_t *offsets, int E, int M,
                      int N, int K, int dtype, void *C, hipStream_t st)
{
    const Fp8Args a = {A, a_scale, a_rows, M_a, W, w_scale, offsets, E, M, N, K,
                       (K + KB8 - 1) / KB8, (N + 127) / 128, (uint16_t *)C};
    return dtype == QG_DT_BF16 ? launch<true>(a, st) : launch<false>(a, st);
}

long long fp8_workgroups(bool grouped, int E, int M, int N, int K)
{
    Fp8Args a = {};
    a.offsets = grouped ? (const int32_t *)1 : nullptr;
    a.E = E;
    a.M = M;
    return row_blocks(a, 64) * ((N + 127) / 128);
}

void describe_fp8(bool grouped, int E, int M, int N, int K, char *buf, size_t n)
{
    snprintf(buf, n, "tiled kernel, 64 x 128");
}

} // namespace qg
