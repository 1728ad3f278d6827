// The steps around a mixture-of-experts layer's grouped product: the choice
// of experts for each token, the sort of the chosen slots by expert, and the
// weighted sum of the experts' rows back to the tokens.
#include "qg_device.h"
#include "qg_launch.h"

namespace qg {
namespace {

__device__ inline float load_as_f32(const void *p, int dtype, size_t i)
{
    if (dtype == QG_DT_F32) return ((const float *)p)[i];
    const uint16_t b = ((const uint16_t *)p)[i];
    return dtype == QG_DT_F16 ? h2f(b) : bf2f(b);
}

// One wave per token; lane l holds experts l, l + 64, ... (VPL of them).
// Everything that decides an order is in 64 bits.
template <int VPL>
__global__ __launch_bounds__(256) void moe_route_kernel(
    const void *__restrict__ logits, int dtype, const float *__restrict__ bias, int T, int E,
    int topk, int n_group, int topk_group, float scaling, unsigned flags,
    int32_t *__restrict__ ids, float *__restrict__ weights)
{
    __shared__ double sh[4][VPL * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x * 4 + wave;
    const bool live = t < T;
    const double NINF = -__builtin_inf();
    double score[VPL], choice[VPL];
    double mx = NINF;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 64 * i;
        double l = NINF;
        if (live && e < E) {
            l = load_as_f32(logits, dtype, (size_t)t * E + e);
            if (l != l) l = NINF;
        }
        score[i] = l;
        mx = l > mx ? l : mx;
    }
    if (!(flags & 1u)) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double m = __shfl_xor(mx, o);
            mx = m > mx ? m : mx;
        }
        double sum = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const double l = score[i];
            const double p = l == NINF ? 0.0 : l == mx ? 1.0 : exp(l - mx);
            choice[i] = l;
            score[i] = p;
            sum += p;
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
        for (int i = 0; i < VPL; ++i) score[i] = sum > 0 ? score[i] / sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            choice[i] = score[i];
            score[i] = 1.0 / (1.0 + exp(-score[i]));
        }
    }
    // without a bias the logits rank as the scores do
    if (bias) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E && choice[i] != NINF) {
                choice[i] = score[i] + (double)bias[e];
                if (choice[i] != choice[i]) choice[i] = NINF;
            }
        }
    }
    if (n_group > 1) {
        const int size = E / n_group;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            sh[wave][lane + 64 * i] = !bias && (flags & 4u) && choice[i] != NINF ? score[i] : choice[i];
        __syncthreads();
        double a = NINF, b = NINF;
        if (lane < n_group) {
            for (int j = 0; j < size; ++j) {
                const double v = sh[wave][lane * size + j];
                if (v > a) { b = a; a = v; }
                else if (v > b) b = v;
            }
        }
        if ((flags & 4u) && b != NINF) a += b;
        int rank = 0;
        for (int g = 0; g < n_group; ++g) {
            const double v = __shfl(a, g);
            rank += v > a || (v == a && g < lane);
        }
        const unsigned long long keep = __ballot(lane < n_group && rank < topk_group);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E && !((keep >> (e / size)) & 1)) choice[i] = NINF;
        }
    }
    double mine = 0;
    int my_id = -1;
    for (int j = 0; j < topk; ++j) {
        double best = NINF, s = 0;
        int id = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (choice[i] > best) {
                best = choice[i];
                s = score[i];
                id = lane + 64 * i;
            }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double ob = __shfl_xor(best, o), os = __shfl_xor(s, o);
            const int oi = __shfl_xor(id, o);
            if (ob > best || (ob == best && oi < id)) {
                best = ob;
                s = os;
                id = oi;
            }
        }
        if (best == NINF) break;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane + 64 * i == id) choice[i] = NINF;
        if (lane == j) {
            mine = s;
            my_id = id;
        }
    }
    double sum = mine;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    double w = mine;
    if (flags & 2u) w = sum > 0 ? w / sum : 0.0;
    if (live && lane < topk) {
        ids[(size_t)t * topk + lane] = my_id;
        weights[(size_t)t * topk + lane] = (float)(w * (double)scaling);
    }
}

// One workgroup: a stable counting sort of n slots by expert.  Wave w takes a
// contiguous run of the slots; lanes with the same expert find their rank by
// comparing ids bit by bit over ballots.
constexpr int SORT_MAX_E = 1024;

__device__ inline unsigned long long same_id(int id, int bits)
{
    unsigned long long m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const unsigned long long v = __ballot((id >> b) & 1);
        m &= ((id >> b) & 1) ? v : ~v;
    }
    return m;
}

__global__ __launch_bounds__(256) void moe_sort_one_kernel(
    const int32_t *__restrict__ ids, int n, int topk, int E, int bits,
    int32_t *__restrict__ offsets, int32_t *__restrict__ row_token, int32_t *__restrict__ slot_row)
{
    __shared__ int cnt[4][SORT_MAX_E + 1];
    __shared__ int tot[SORT_MAX_E + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < 4 * (SORT_MAX_E + 1); i += 256) (&cnt[0][0])[i] = 0;
    __syncthreads();
    const int run = ((n + 255) / 256) * 64;
    const int s0 = wave * run, s1 = s0 + run < n ? s0 + run : n;
    for (int s = s0 + lane; s < s1; s += 64) {
        const int id = ids[s];
        if (id >= 0 && id < E) atomicAdd(&cnt[wave][id], 1);
    }
    __syncthreads();
    for (int e = tid; e < E; e += 256) {
        int a = 0;
        for (int w = 0; w < 4; ++w) {
            const int c = cnt[w][e];
            cnt[w][e] = a;
            a += c;
        }
        tot[e] = a;
    }
    __syncthreads();
    if (tid == 0) {
        int a = 0;
        for (int e = 0; e < E; ++e) {
            const int c = tot[e];
            tot[e] = a;
            a += c;
        }
        tot[E] = a;
    }
    __syncthreads();
    for (int e = tid; e <= E; e += 256) offsets[e] = tot[e];
    const unsigned long long below = (1ull << lane) - 1;
    for (int sb = s0; sb < s1; sb += 64) {
        const int s = sb + lane;
        int id = s < s1 ? ids[s] : E;
        if (id < 0 || id > E) id = E;
        const unsigned long long m = same_id(id, bits);
        int row = -1;
        if (id < E) row = tot[id] + cnt[wave][id] + __popcll(m & below);
        __builtin_amdgcn_wave_barrier();
        if (id < E && (m & below) == 0) cnt[wave][id] += __popcll(m);
        __builtin_amdgcn_wave_barrier();
        if (s < s1) {
            slot_row[s] = row;
            if (row >= 0) row_token[row] = s / topk;
        }
    }
}

__global__ __launch_bounds__(256) void moe_combine_kernel(
    const uint16_t *__restrict__ Y, int bf16, const int32_t *__restrict__ slot_row,
    const float *__restrict__ weights, int topk, int M_rows, int N, uint16_t *__restrict__ out)
{
    const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float a = 0.f;
    for (int j = 0; j < topk; ++j) {
        const int r = slot_row[(size_t)t * topk + j];
        if (r < 0 || r >= M_rows) continue;
        const uint16_t y = Y[(size_t)r * N + n];
        a = __builtin_fmaf(weights[(size_t)t * topk + j], bf16 ? bf2f(y) : h2f(y), a);
    }
    out[(size_t)t * N + n] = bf16 ? f2bf(a) : f2h(a);
}

} // namespace

hipError_t launch_moe_route(const void *logits, int dtype, const float *bias, int T, int E,
                            int topk, int n_group, int topk_group, float scaling, unsigned flags,
                            int32_t *ids, float *weights, hipStream_t st)
{
    const dim3 grid((T + 3) / 4), block(256);
#define QG_ROUTE(VPL) \
    hipLaunchKernelGGL((moe_route_kernel<VPL>), grid, block, 0, st, logits, dtype, bias, T, E, topk, \
                       n_group, topk_group, scaling, flags, ids, weights)
    if (E <= 64) QG_ROUTE(1);
    else if (E <= 128) QG_ROUTE(2);
    else if (E <= 256) QG_ROUTE(4);
    else if (E <= 512) QG_ROUTE(8);
    else QG_ROUTE(16);
#undef QG_ROUTE
    return hipGetLastError();
}

size_t moe_sort_workspace_bytes(int T, int topk, int E) { return 0; }

hipError_t launch_moe_sort(const int32_t *ids, int T, int topk, int E, int32_t *offsets,
                           int32_t *row_token, int32_t *slot_row, void *ws, hipStream_t st)
{
    int bits = 1;
    while ((1 << bits) <= E) ++bits;
    hipLaunchKernelGGL(moe_sort_one_kernel, dim3(1), dim3(256), 0, st, ids, T * topk, topk, E, bits,
                       offsets, row_token, slot_row);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void *Y, int dtype, const int32_t *slot_row,
                              const float *weights, int T, int topk, int M_rows, int N, void *out,
                              hipStream_t st)
{
    // blockIdx.y carries 16 bits' worth of tokens at most
    for (int t0 = 0; t0 < T; t0 += 65535) {
        const int n = T - t0 < 65535 ? T - t0 : 65535;
        hipLaunchKernelGGL(moe_combine_kernel, dim3((N + 255) / 256, n), dim3(256), 0, st,
                           (const uint16_t *)Y, dtype == QG_DT_BF16, slot_row + (size_t)t0 * topk,
                           weights + (size_t)t0 * topk, topk, M_rows, N,
                           (uint16_t *)out + (size_t)t0 * N);
    }
    return hipGetLastError();
}

} // namespace qg
