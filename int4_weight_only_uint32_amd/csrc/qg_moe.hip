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

// ---- routing ----
// One wave per token; lane l holds the VPL experts from l * VPL on.  The answer is
// the order of choices in 64 bits.  Taken there for every expert, the exponentials
// alone cost 59 us for 16384 tokens of 256 experts (18 MB, 4 us at the memory's
// rate), so the order is first taken in 32 bits, with a bound on how far each
// choice may be off: where two neighbours among the chosen (or the group
// values at the border) are closer than both their bounds, and only there, the
// wave does the token again in 64.  Without a bias the logits rank as the scores
// do, and exactly.  That case takes 17 us, 14 of them the issue of 539 vector
// instructions a token, 1.5 the tokens done again.
struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int dtype, T, E, topk, n_group, topk_group;
    float scaling;
    unsigned flags;
};
constexpr unsigned ROUTE_SIGMOID = 1u, ROUTE_RENORMALIZE = 2u, ROUTE_GROUP_TOP2 = 4u;

// x of the lanes of a wave, and the largest of all in every lane.
__device__ inline unsigned wave_max(unsigned x)
{
#define QG_DPP_MAX(ctrl, rows) \
    x = __builtin_elementwise_max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xf, false))
    QG_DPP_MAX(0x111, 0xf);      // 1, 2, 4, 8 lanes down within a row of 16
    QG_DPP_MAX(0x112, 0xf);
    QG_DPP_MAX(0x114, 0xf);
    QG_DPP_MAX(0x118, 0xf);
    QG_DPP_MAX(0x142, 0xa);      // a row's last lane to the next row
    QG_DPP_MAX(0x143, 0xc);      // the second row's last lane to the upper half
#undef QG_DPP_MAX
    return (unsigned)__builtin_amdgcn_readlane((int)x, 63);
}

// The sum over a wave, in every lane.
__device__ inline float wave_sum(float x)
{
#define QG_DPP_ADD(ctrl, rows) \
    x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, rows, 0xf, false))
    QG_DPP_ADD(0x111, 0xf);
    QG_DPP_ADD(0x112, 0xf);
    QG_DPP_ADD(0x114, 0xf);
    QG_DPP_ADD(0x118, 0xf);
    QG_DPP_ADD(0x142, 0xa);
    QG_DPP_ADD(0x143, 0xc);
#undef QG_DPP_ADD
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// Floats as unsigned words of the same order (both zeros alike; 0 is below
// every value).
__device__ inline unsigned order_key(float x)
{
    const unsigned b = __builtin_bit_cast(unsigned, x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ inline float key_value(unsigned k)
{
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ inline float sigmoid_near(float l)
{
    // (clamped: beyond, the result is under 2^-120, and weights like that are taken in 64 bits)
    const float x = __builtin_fminf(__builtin_fmaxf(-l, -87.0f), 87.0f);
    return rcp_near(1.0f + exp_near(x));
}

// The chosen experts' scores to weights; lane j holds the j-th.
__device__ inline void route_store(const RouteArgs &a, int t, int lane, int id, float w)
{
    if (lane < a.topk) {
        a.ids[(size_t)t * a.topk + lane] = id;
        a.weights[(size_t)t * a.topk + lane] = w;
    }
}

// A token in 64 bits throughout.  sh: this wave's VPL * 64 doubles.
template <int VPL>
__device__ inline void route_exact(const RouteArgs &a, int t, double *sh)
{
    const int lane = threadIdx.x & 63;
    const double NINF = -__builtin_inf();
    double score[VPL], choice[VPL];
    double mx = NINF;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        double l = NINF;
        if (e < a.E) {
            l = load_as_f32(a.logits, a.dtype, (size_t)t * a.E + e);
            if (l != l) l = NINF;
        }
        score[i] = choice[i] = l;
        mx = l > mx ? l : mx;
    }
    if (!(a.flags & ROUTE_SIGMOID)) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double m = __shfl_xor(mx, o);
            mx = m > mx ? m : mx;
        }
        double sum = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const double l = score[i];
            score[i] = l == NINF ? 0.0 : l == mx ? 1.0 : exp(l - mx);
            sum += score[i];
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
        for (int i = 0; i < VPL; ++i) score[i] = sum > 0 ? score[i] / sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) score[i] = 1.0 / (1.0 + exp(-score[i]));
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane * VPL + i;
            if (e < a.E && choice[i] != NINF) {
                choice[i] = score[i] + (double)a.bias[e];
                if (choice[i] != choice[i]) choice[i] = NINF;
            }
        }
    }
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        const bool sums = (a.flags & ROUTE_GROUP_TOP2) != 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            sh[lane * VPL + i] = !a.bias && sums && choice[i] != NINF ? score[i] : choice[i];
        // the wave's own words only, in order: no other wave to wait for
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        debug_stage_sync();
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        double v = NINF, v2 = NINF;
        if (lane < a.n_group) {
            int j = 0;
            for (; j + 8 <= size; j += 8) {      // eight reads in flight
                double x[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = sh[lane * size + j + u];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    v2 = __builtin_fmax(v2, __builtin_fmin(v, x[u]));
                    v = __builtin_fmax(v, x[u]);
                }
            }
            for (; j < size; ++j) {
                const double x = sh[lane * size + j];
                v2 = __builtin_fmax(v2, __builtin_fmin(v, x));
                v = __builtin_fmax(v, x);
            }
        }
        if (sums && v2 != NINF) v += v2;
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double x = __shfl(v, g);
            rank += x > v || (x == v && g < lane);
        }
        const unsigned long long keep = __ballot(lane < a.n_group && rank < a.topk_group);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int e = lane * VPL + i;
            if (e < a.E && !((keep >> (e / size)) & 1)) choice[i] = NINF;
        }
    }
    // keys of the same order as the choices (0 for a masked expert); the largest of
    // the wave by its upper words, then by the lower ones of those that have it
    unsigned long long key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const unsigned long long b = __builtin_bit_cast(unsigned long long, choice[i] + 0.0);
        key[i] = choice[i] == NINF ? 0ull : (b >> 63) ? ~b : b | (1ull << 63);
    }
    double mine = 0;
    int my_id = -1;
    for (int j = 0; j < a.topk; ++j) {
        unsigned long long best = 0;
        double s = 0;
        int id = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                s = score[i];
                id = lane * VPL + i;
            }
        const unsigned hi = wave_max((unsigned)(best >> 32));
        if (hi == 0) break;
        const bool has = (unsigned)(best >> 32) == hi;
        const unsigned lo = wave_max(has ? (unsigned)best : 0u);
        const int owner = __builtin_ctzll(__ballot(has && (unsigned)best == lo));
        const long long sb = __builtin_bit_cast(long long, s);
        const unsigned s_lo = (unsigned)__builtin_amdgcn_readlane((int)sb, owner);
        const unsigned s_hi = (unsigned)__builtin_amdgcn_readlane((int)(sb >> 32), owner);
        id = __builtin_amdgcn_readlane(id, owner);
        if (lane == j) {
            mine = __builtin_bit_cast(double, (unsigned long long)s_hi << 32 | s_lo);
            my_id = id;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = lane * VPL + i == id ? 0ull : key[i];
    }
    double sum = mine;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    double w = mine;
    if (a.flags & ROUTE_RENORMALIZE) w = sum > 0 ? w / sum : 0.0;
    route_store(a, t, lane, my_id, (float)(w * (double)a.scaling));
}

// How far a choice c in 32 bits may be from its value, at most: the score's error
// and the rounding of its sum with the bias (half a step, 2^-24 |c|; the rest of
// 1.0625 is for the roundings of the bound itself).  The scores' errors, in units of 2^-24:
//   sigmoid, s = 1 / d, d = 1 + e: e is off by 4 e (exp_near), which is 4 s (1 - s) of s;
//   d by half a step, 1 for d < 2, which is s^2; the reciprocal by a step, 1 under
//   s = 1: together at most 2.34, at s = 2/3, and less under 1/2.  Taken as 4, 2^-22.
//   softmax, p = e / sum: e is off by 4 e and |l - max| e (its argument's rounding);
//   the sum by 4, by 22 roundings (16 experts a lane, six joins) and by the mean of
//   |l - max|, which is at most ln 1024 < 7 (entropy); p by 2 (reciprocal) and 1; and p |l - max|
//   is under 0.4: 41 in all.  Taken as 64, 2^-18.
__device__ inline float route_error(bool sigmoid, float c)
{
    return (sigmoid ? 0x1p-22f : 0x1p-18f) + 0x1.1p-24f * __builtin_fabsf(c);
}

template <int VPL>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a, int wide, int gl_shift, int size, int size_magic)
{
    __shared__ double sh[4][VPL * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x * 4 + wave;
    if (t >= a.T) return;
    const bool sigmoid = (a.flags & ROUTE_SIGMOID) != 0, sums = (a.flags & ROUTE_GROUP_TOP2) != 0;
    const bool renorm = (a.flags & ROUTE_RENORMALIZE) != 0;
    const float NINF = -__builtin_inff();
    const int e0 = lane * VPL;
    const size_t at = (size_t)t * a.E + e0;

    float l[VPL], b[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        l[i] = NINF;
        b[i] = 0.f;
    }
    if (wide) {          // whole vectors: E a multiple of VPL, rows and bias aligned
        typedef float fvec __attribute__((ext_vector_type(VPL)));
        typedef uint16_t hvec __attribute__((ext_vector_type(VPL)));
        if (e0 < a.E) {
            if (a.dtype == QG_DT_F32) {
                const fvec v = *reinterpret_cast<const fvec *>((const float *)a.logits + at);
#pragma unroll
                for (int i = 0; i < VPL; ++i) l[i] = v[i];
            } else {
                const hvec v = *reinterpret_cast<const hvec *>((const uint16_t *)a.logits + at);
#pragma unroll
                for (int i = 0; i < VPL; ++i) l[i] = a.dtype == QG_DT_F16 ? h2f(v[i]) : bf2f(v[i]);
            }
            if (a.bias) {
                const fvec v = *reinterpret_cast<const fvec *>(a.bias + e0);
#pragma unroll
                for (int i = 0; i < VPL; ++i) b[i] = v[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e0 + i < a.E) {
                l[i] = load_as_f32(a.logits, a.dtype, at + i);
                if (a.bias) b[i] = a.bias[e0 + i];
            }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = l[i] != l[i] ? NINF : l[i];

    // The choices c and what the groups are valued by (v): the logits where they
    // rank as the scores do, else the scores (plus bias).
    const bool scored = a.bias || (a.n_group > 1 && sums);
    float c[VPL], v[VPL], mx = 0.f, inv = 1.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = v[i] = l[i];
    if (!sigmoid) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = __builtin_elementwise_max(m, order_key(l[i]));
        mx = key_value(wave_max(m));
    }
    auto exp_of = [&](float x) {
        const float e = exp_near(__builtin_fmaxf(x - mx, -150.0f));     // (NaN to -150: x = mx = +-infinity)
        return x == mx ? 1.0f : e;
    };
    if (scored || (!sigmoid && !renorm)) {
        float sc[VPL];
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) sc[i] = sigmoid_near(l[i]);
        } else {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float e = exp_of(l[i]);
                sc[i] = l[i] > NINF ? e : 0.f;
                sum += sc[i];
            }
            sum = wave_sum(sum);
            inv = sum > 0.f ? rcp_near(sum) : 0.f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) sc[i] *= inv;
        }
        if (scored) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const float x = sc[i] + b[i];     // (b is 0 without a bias)
                const float y = l[i] > NINF && x == x ? x : NINF;
                v[i] = y;
                c[i] = a.bias ? y : c[i];
            }
        }
    }
    bool unsure = false;
    unsigned keep = ~0u;       // bit i: this lane's expert i is in a group that stays
    if (a.n_group > 1) {
        // The two largest values of each group.  Groups on whole runs of a power of
        // two lanes (gl_shift >= 0): in all lanes of the run, by exchanges; others: in
        // lane g for group g, out of LDS.
        float v1 = NINF, v2 = NINF;
        int mine = lane, stride = 0;       // this lane's group, its first lane's shift
        if (gl_shift >= 0) {
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                v2 = __builtin_fmaxf(v2, __builtin_fminf(v1, v[i]));
                v1 = __builtin_fmaxf(v1, v[i]);
            }
            for (int o = 0; o < gl_shift; ++o) {
                const float u = __shfl_xor(v1, 1 << o), u2 = __shfl_xor(v2, 1 << o);
                v2 = __builtin_fmaxf(__builtin_fminf(v1, u), __builtin_fmaxf(v2, u2));
                v1 = __builtin_fmaxf(v1, u);
            }
            mine = lane >> gl_shift;
            stride = gl_shift;
        } else {
            float *vals = reinterpret_cast<float *>(sh[wave]);
#pragma unroll
            for (int i = 0; i < VPL; ++i) vals[e0 + i] = v[i];
            // (the wave's own words, in order: no other wave to wait for)
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            debug_stage_sync();
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (lane < a.n_group)
                for (int j = 0; j < size; ++j) {
                    const float x = vals[lane * size + j];
                    v2 = __builtin_fmaxf(v2, __builtin_fminf(v1, x));
                    v1 = __builtin_fmaxf(v1, x);
                }
            debug_stage_sync();
            __builtin_amdgcn_wave_barrier();
        }
        const bool group = mine < a.n_group;
        auto group_value = [&](int g) {
            return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v1), g << stride));
        };
        bool stays;
        if (scored) {
            // twice the largest error of a value, so that values further apart
            // than it are in order
            float tol = 0.f;
            if (sums && v2 > NINF) {
                tol = route_error(sigmoid, v1) + route_error(sigmoid, v2) + 0x1.1p-24f * __builtin_fabsf(v1 + v2);
                v1 += v2;
            } else if (v1 > NINF) {
                tol = route_error(sigmoid, v1);
            }
            tol = 2.f * __builtin_bit_cast(float, wave_max(__builtin_bit_cast(unsigned, tol)));
            const float hi = v1 + tol, lo = v1 - tol;
            int above = 0, not_below = -1;      // (its own value is not below it)
            for (int g = 0; g < a.n_group; ++g) {
                const float x = group_value(g);
                above += x > hi;
                not_below += x >= lo;
            }
            // (sums past binary32's range, or an infinite bias: no order without 64 bits)
            unsure = !(tol < __builtin_inff()) || __ballot(group && above < a.topk_group && not_below >= a.topk_group) != 0;
            stays = not_below < a.topk_group;
        } else {
            int before = 0;
            for (int g = 0; g < a.n_group; ++g) {
                const float x = group_value(g);
                before += x > v1 || (x == v1 && g < mine);
            }
            stays = before < a.topk_group;
        }
        stays = stays && group;
        if (gl_shift >= 0) {
            keep = stays ? ~0u : 0u;
        } else {
            const unsigned long long groups = __ballot(stays);
            keep = 0;
            // e / size for e < 1024 as e * ceil(2^20 / size) >> 20: off by less than
            // 1024 / 2^20 of the quotient, and size is at most 512
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                keep |= (unsigned)((groups >> (((e0 + i) * size_magic >> 20) & 63)) & 1) << i;
        }
    }
    // Each lane's keys (0 for a masked expert) in descending order, the lower
    // index first among equals (neighbours change places only if out of order),
    // four bits of the index of each in one word; then the largest head of the
    // wave, topk times.
    unsigned key[VPL], idx[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = (keep >> i & 1) && c[i] > NINF ? order_key(c[i]) : 0u;
        idx[i] = i;
    }
#pragma unroll
    for (int k = 0; k < VPL; ++k)
#pragma unroll
        for (int i = k & 1; i + 1 < VPL; i += 2) {
            const bool swap = key[i] < key[i + 1];
            const unsigned big = __builtin_elementwise_max(key[i], key[i + 1]);
            key[i + 1] = __builtin_elementwise_min(key[i], key[i + 1]);
            key[i] = big;
            const unsigned x = idx[i];
            idx[i] = swap ? idx[i + 1] : x;
            idx[i + 1] = swap ? x : idx[i + 1];
        }
    unsigned order[VPL > 8 ? 2 : 1] = {};
#pragma unroll
    for (int i = 0; i < VPL; ++i) order[i / 8] |= idx[i] << (4 * (i & 7));
    int my_id = -1, found = 0;
    float my_c = 0.f;
    // with a bias one more than topk, to see that the last chosen is clear of it
    const int rounds = a.topk + (a.bias != nullptr ? 1 : 0);
    uint2v *heads = reinterpret_cast<uint2v *>(sh[wave]);     // (at most VPL * 64 are found)
    if (!unsure) {
        for (; found < rounds; ++found) {
            const unsigned m = wave_max(key[0]);
            if (m == 0) break;
            const int owner = __builtin_ctzll(__ballot(key[0] == m));
            if (lane == owner) {
                heads[found] = uint2v{m, (unsigned)e0 + (order[0] & 15)};
#pragma unroll
                for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
                key[VPL - 1] = 0;
                order[0] >>= 4;
                if (VPL > 8) {
                    order[0] |= order[VPL > 8] << 28;
                    order[VPL > 8] >>= 4;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        debug_stage_sync();
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (lane < found) {
            const uint2v h = heads[lane];
            my_c = key_value(h.x);
            my_id = (int)h.y;
        }
    }
    if (a.bias) {
        const float after = __shfl_down(my_c, 1);
        const bool clear = my_c - after > route_error(sigmoid, my_c) + route_error(sigmoid, after);
        unsure = unsure || __ballot(lane + 1 < found && !clear) != 0;
    }
    if (lane >= a.topk) my_id = -1;
    // weights from the chosen logits
    float s = 0.f;
    if (!unsure && my_id >= 0) {
        const float x = load_as_f32(a.logits, a.dtype, (size_t)t * a.E + my_id);
        s = sigmoid ? sigmoid_near(x) : exp_of(x) * inv;
    }
    const float sum = wave_sum(s);
    // weights that run out of 32 bits: in 64
    if (__ballot(my_id >= 0 && s < 0x1p-120f)) unsure = true;
    if (unsure) {
        route_exact<VPL>(a, t, sh[wave]);
        return;
    }
    float w = s * a.scaling;
    if (renorm) w = sum > 0.f ? s / sum * a.scaling : 0.f;
    route_store(a, t, lane, my_id, w);
}

// ---- sort ----
// A stable counting sort of the slots by expert, bound by latency: 16383 x 8 slots
// are 1.6 MB in and out, 0.3 us at the memory's rate.  A workgroup of SORT_WAVES
// waves takes a run of slots, each wave a contiguous part of it.  Counts per wave
// and expert stand in LDS; in the pass that places the slots, the lanes of a
// wave that hold the same expert find each other by ballots over the id's
// bits, so a slot's rank is a count of lower lanes and no order of atomics
// decides anything.  Few slots: one workgroup, one launch.  More: one launch
// counts each workgroup's slots per expert, the next adds the counts of the
// workgroups before it (each for itself, up to 256 rows of E counts).
constexpr int SORT_MAX_E = 1024, SORT_WAVES = 8, SORT_THREADS = 64 * SORT_WAVES;
// Slots up to which one workgroup does it all, of 8 waves, or for up to 512 experts (whose
// counts of 16 waves LDS holds) of 16 from 1025 slots on.  In a graph: 1024 slots of 256
// experts 4.3 us (8 waves) and 4.5 (16), 2000 of 64 5.9 and 5.3, with two launches 6.3;
// 4000 7.0 (16 waves) and 6.5 (two launches), which outside a graph are the host's 10.6.
constexpr int SORT_ONE = 2048, SORT_ONE_WIDE = 4096, SORT_WIDE_E = 512, SORT_WIDE_FROM = 1024;
constexpr int SORT_MAX_WGS = 256;

// Per-wave counts of this workgroup's slots [s0, s1), run slots to a wave.
template <int WAVES, int MAX_E>
__device__ inline void sort_count(const int32_t *__restrict__ ids, int s0, int s1, int run, int E,
                                  int (&cnt)[WAVES][MAX_E])
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int w = 0; w < WAVES; ++w)
        for (int e = tid; e < E; e += 64 * WAVES) cnt[w][e] = 0;
    __syncthreads();
    const int a = s0 + wave * run, b = a + run < s1 ? a + run : s1;
#pragma unroll 4
    for (int s = a + lane; s < b; s += 64) {
        const int id = ids[s];
        if (id >= 0 && id < E) atomicAdd(&cnt[wave][id], 1);
    }
    __syncthreads();
}

// Exclusive prefix over the experts of the totals, two of them a thread; out[E]
// is the sum.  Every thread of the workgroup calls it.
template <int WAVES>
__device__ inline void sort_scan(int (&sums)[WAVES], int E, const int *tot, int *out)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e = 2 * tid;
    const int t0 = e < E ? tot[e] : 0, t1 = e + 1 < E ? tot[e + 1] : 0;
    int x = t0 + t1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(x, o);
        if (lane >= o) x += v;
    }
    if (lane == 63) sums[wave] = x;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        if (w < wave) before += sums[w];
    const int at = before + x - t0 - t1;
    if (e <= E) out[e] = at;
    if (e + 1 <= E) out[e + 1] = at + t0;
    if (tid == 64 * WAVES - 1 && E == 128 * WAVES) out[E] = at + t0 + t1;
    __syncthreads();
}

// Places the workgroup's slots: cnt[w][e] is the row of wave w's next slot of e.
template <int WAVES, int MAX_E>
__device__ inline void sort_place(const int32_t *__restrict__ ids, int s0, int s1, int run, int topk,
                                  int E, int bits, int (&cnt)[WAVES][MAX_E],
                                  int32_t *__restrict__ row_token, int32_t *__restrict__ slot_row)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int a = s0 + wave * run, b = a + run < s1 ? a + run : s1;
    const unsigned long long below = (1ull << lane) - 1;
    volatile int *next = cnt[wave];
    int ahead = a + lane < b ? ids[a + lane] : -1;
    for (int sb = a; sb < b; sb += 64) {
        const int s = sb + lane;
        const int raw = ahead;
        ahead = s + 64 < b ? ids[s + 64] : -1;
        const int id = raw >= 0 && raw < E ? raw : E;
        unsigned long long same = ~0ull;
        for (int k = 0; k < bits; ++k) {
            const bool one = (id >> k) & 1;
            const unsigned long long v = __ballot(one);
            same &= one ? v : ~v;
        }
        // the wave's LDS accesses are in order: all lanes read their count
        // before the lowest lane of each expert raises it
        int row = -1;
        if (id < E) row = next[id] + __popcll(same & below);
        debug_stage_sync();
        __builtin_amdgcn_wave_barrier();
        if (id < E && (same & below) == 0) next[id] = row + __popcll(same);
        debug_stage_sync();
        __builtin_amdgcn_wave_barrier();
        if (s < b) {
            slot_row[s] = row;
            if (row >= 0) row_token[row] = s / topk;
        }
    }
}

template <int WAVES, int MAX_E>
__global__ __launch_bounds__(64 * WAVES) void moe_sort_one_kernel(
    const int32_t *__restrict__ ids, int n, int run, int topk, int E, int bits,
    int32_t *__restrict__ offsets, int32_t *__restrict__ row_token, int32_t *__restrict__ slot_row)
{
    __shared__ int cnt[WAVES][MAX_E];
    __shared__ int tot[MAX_E], first[MAX_E + 1], sums[WAVES];
    const int tid = threadIdx.x;
    sort_count(ids, 0, n, run, E, cnt);
    for (int e = tid; e < E; e += 64 * WAVES) {
        int a = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) a += cnt[w][e];
        tot[e] = a;
    }
    __syncthreads();
    sort_scan(sums, E, tot, first);
    for (int e = tid; e <= E; e += 64 * WAVES) {
        int at = first[e];
        offsets[e] = at;
        if (e < E)
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const int c = cnt[w][e];
                cnt[w][e] = at;
                at += c;
            }
    }
    __syncthreads();
    sort_place(ids, 0, n, run, topk, E, bits, cnt, row_token, slot_row);
}

// hist [workgroups, E], rows of whole 16-byte words, zeros behind E
__device__ inline int hist_stride(int E) { return (E + 3) & ~3; }

__global__ __launch_bounds__(SORT_THREADS) void moe_sort_count_kernel(
    const int32_t *__restrict__ ids, int n, int run, int E, int32_t *__restrict__ hist)
{
    __shared__ int cnt[SORT_WAVES][SORT_MAX_E];
    const int s0 = blockIdx.x * (run * SORT_WAVES);
    const int s1 = n - s0 < run * SORT_WAVES ? n : s0 + run * SORT_WAVES;
    sort_count(ids, s0, s1, run, E, cnt);
    const int stride = hist_stride(E);
    for (int e = threadIdx.x; e < stride; e += SORT_THREADS) {
        int a = 0;
        if (e < E)
#pragma unroll
            for (int w = 0; w < SORT_WAVES; ++w) a += cnt[w][e];
        hist[(size_t)blockIdx.x * stride + e] = a;
    }
}

__global__ __launch_bounds__(SORT_THREADS) void moe_sort_place_kernel(
    const int32_t *__restrict__ ids, int n, int run, int topk, int E, int bits,
    const int32_t *__restrict__ hist, int32_t *__restrict__ offsets, int32_t *__restrict__ row_token,
    int32_t *__restrict__ slot_row)
{
    __shared__ int cnt[SORT_WAVES][SORT_MAX_E];
    __shared__ int tot[SORT_MAX_E], before[SORT_MAX_E], first[SORT_MAX_E + 1], sums[SORT_WAVES];
    constexpr int BATCH = 16;
    const int tid = threadIdx.x, wgs = gridDim.x, me = blockIdx.x;
    const int s0 = me * (run * SORT_WAVES);
    const int s1 = n - s0 < run * SORT_WAVES ? n : s0 + run * SORT_WAVES;
    const int stride = hist_stride(E), quads = stride / 4;
    for (int e = tid; e < stride; e += SORT_THREADS) tot[e] = before[e] = 0;
    __syncthreads();
    // The counts of all workgroups, four experts a thread; the threads that these leave
    // over share the rows, and a thread's loads are in flight together (they come from
    // other XCDs)
    const int span = quads > 1 ? 1 << (32 - __builtin_clz(quads - 1)) : 1;      // at most 256
    const int parts = SORT_THREADS / span, part = tid / span, quad = tid - part * span;
    if (quad < quads) {
        int4v all = {0, 0, 0, 0}, mine = all;
        for (int w0 = part; w0 < wgs; w0 += BATCH * parts) {
            int4v c[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int w = w0 + u * parts;      // (past the end: the last row again, not counted)
                c[u] = reinterpret_cast<const int4v *>(hist)[(w < wgs ? w : wgs - 1) * quads + quad];
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int w = w0 + u * parts;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    all[x] += w < wgs ? c[u][x] : 0;
                    mine[x] += w < me ? c[u][x] : 0;
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            atomicAdd(&tot[quad * 4 + x], all[x]);
            atomicAdd(&before[quad * 4 + x], mine[x]);
        }
    }
    sort_count(ids, s0, s1, run, E, cnt);      // (its barriers publish tot and before)
    sort_scan(sums, E, tot, first);
    for (int e = tid; e <= E; e += SORT_THREADS) {
        if (me == 0) offsets[e] = first[e];
        if (e < E) {
            int at = first[e] + before[e];
#pragma unroll
            for (int w = 0; w < SORT_WAVES; ++w) {
                const int c = cnt[w][e];
                cnt[w][e] = at;
                at += c;
            }
        }
    }
    __syncthreads();
    sort_place(ids, s0, s1, run, topk, E, bits, cnt, row_token, slot_row);
}

// ---- combine ----
// One workgroup of 256 lanes per token and run of columns; a lane holds 8 columns
// (16 bytes).  A token's rows and weights are the same for all lanes (scalar
// loads); the loads of eight rows are in flight before the first is used.
// Bound by memory: topk rows read for one written (4093 x 8 rows of 7168 bf16: 92 us,
// 5.7 TB/s).
template <bool BF16>
__device__ inline float in16(unsigned b) { return BF16 ? bf2f((uint16_t)b) : h2f((uint16_t)b); }

template <bool BF16>
__device__ inline unsigned out_pair(float a, float b)
{
    return BF16 ? f2bf(a) | (unsigned)f2bf(b) << 16 : f2h(a) | (unsigned)f2h(b) << 16;
}

template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_kernel(
    const uint16_t *__restrict__ Y, const int32_t *__restrict__ slot_row,
    const float *__restrict__ weights, int topk, int M_rows, int N, uint16_t *__restrict__ out)
{
    const int t = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (n >= N) return;
    const int32_t *row = slot_row + (size_t)t * topk;
    const float *wt = weights + (size_t)t * topk;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < topk; j0 += 8) {
        uint4v y[8];
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = j0 + j < topk ? row[j0 + j] : -1;
            y[j] = uint4v{0u, 0u, 0u, 0u};
            w[j] = 0.f;
            if (r >= 0 && r < M_rows) {
                w[j] = wt[j0 + j];
                y[j] = __builtin_nontemporal_load(reinterpret_cast<const uint4v *>(Y + (size_t)r * N + n));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] = __builtin_fmaf(w[j], in16<BF16>(y[j][i]), acc[2 * i]);
                acc[2 * i + 1] = __builtin_fmaf(w[j], in16<BF16>(y[j][i] >> 16), acc[2 * i + 1]);
            }
    }
    uint4v o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = out_pair<BF16>(acc[2 * i], acc[2 * i + 1]);
    __builtin_nontemporal_store(o, reinterpret_cast<uint4v *>(out + (size_t)t * N + n));
}

// Rows that are no whole 16-byte words, or stand at such an address: one
// column a lane.
template <bool BF16>
__global__ __launch_bounds__(256) void moe_combine_narrow_kernel(
    const uint16_t *__restrict__ Y, const int32_t *__restrict__ slot_row,
    const float *__restrict__ weights, int topk, int M_rows, int N, uint16_t *__restrict__ out)
{
    const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float a = 0.f;
    for (int j = 0; j < topk; ++j) {
        const int r = slot_row[(size_t)t * topk + j];
        if (r < 0 || r >= M_rows) continue;
        a = __builtin_fmaf(weights[(size_t)t * topk + j], in16<BF16>(Y[(size_t)r * N + n]), a);
    }
    out[(size_t)t * N + n] = BF16 ? f2bf(a) : f2h(a);
}

} // namespace

namespace {
template <int VPL>
hipError_t launch_route(const RouteArgs &a, hipStream_t st)
{
    const dim3 grid((a.T + 3) / 4), block(256);
    const int size = a.E / a.n_group, gl = size / VPL;
    const size_t bytes = (size_t)VPL * (a.dtype == QG_DT_F32 ? 4 : 2);
    const int wide = a.E % VPL == 0 && (uintptr_t)a.logits % bytes == 0 && (uintptr_t)a.bias % (VPL * 4) == 0;
    int shift = 0;
    while ((1 << shift) < gl) ++shift;
    if (size % VPL != 0 || (1 << shift) != gl) shift = -1;
    hipLaunchKernelGGL((moe_route_kernel<VPL>), grid, block, 0, st, a, wide, shift, size, ((1 << 20) + size - 1) / size);
    return hipGetLastError();
}
} // namespace

hipError_t launch_moe_route(const void *logits, int dtype, const float *bias, int T, int E,
                            int topk, int n_group, int topk_group, float scaling, unsigned flags,
                            int32_t *ids, float *weights, hipStream_t st)
{
    const RouteArgs a = {logits, bias, ids, weights, dtype, T, E, topk, n_group, topk_group, scaling, flags};
    if (E <= 64) return launch_route<1>(a, st);
    if (E <= 128) return launch_route<2>(a, st);
    if (E <= 256) return launch_route<4>(a, st);
    if (E <= 512) return launch_route<8>(a, st);
    return launch_route<16>(a, st);
}

namespace {
// Slots of one wave (a multiple of 64) of several workgroups: 512 slots
// to a workgroup, or 1024 where the counts of all that every workgroup reads
// would be many; no more than 256 workgroups.  2000 x 8 slots of 128 experts: 7.3 us
// (1024 a workgroup: 8.1, 2048: 9.6), 10000 x 8 of 67: 7.6 (8.3, 9.9), 16383 x 8 of
// 256: 10.5 (9.2, 10.9), 12000 x 6 of 384: 11.1 (10.6, 10.9).
int sort_run(long long n, int E)
{
    const long long least = (n + SORT_THREADS - 1) / SORT_THREADS * E <= 24576 ? 64 : 128;
    const long long per = (n + (long long)SORT_MAX_WGS * SORT_THREADS - 1) / ((long long)SORT_MAX_WGS * SORT_THREADS) * 64;
    return (int)(per < least ? least : per);
}
int sort_wgs(long long n, int E)
{
    if (n <= (E <= SORT_WIDE_E ? SORT_ONE_WIDE : SORT_ONE)) return 1;
    const long long per = (long long)sort_run(n, E) * SORT_WAVES;
    return (int)((n + per - 1) / per);
}
} // namespace

size_t moe_sort_workspace_bytes(int T, int topk, int E)
{
    const long long n = (long long)T * topk;
    const int wgs = sort_wgs(n, E);
    return wgs == 1 ? 0 : W4A16_WS_COUNTER_BYTES + (size_t)wgs * ((E + 3) & ~3) * sizeof(int32_t);
}

hipError_t launch_moe_sort(const int32_t *ids, int T, int topk, int E, int32_t *offsets,
                           int32_t *row_token, int32_t *slot_row, void *ws, hipStream_t st)
{
    int bits = 1;
    while ((1 << bits) <= E) ++bits;     // ids 0 .. E, E for a dropped slot
    const int n = T * topk, wgs = sort_wgs(n, E);
    if (wgs == 1) {
#define QG_SORT_ONE(WAVES, MAX_E) \
    hipLaunchKernelGGL((moe_sort_one_kernel<WAVES, MAX_E>), dim3(1), dim3(64 * WAVES), 0, st, ids, n, \
                       (n + 64 * WAVES - 1) / (64 * WAVES) * 64, topk, E, bits, offsets, row_token, slot_row)
        if (E <= SORT_WIDE_E && n > SORT_WIDE_FROM) QG_SORT_ONE(16, SORT_WIDE_E);
        else QG_SORT_ONE(SORT_WAVES, SORT_MAX_E);
#undef QG_SORT_ONE
        return hipGetLastError();
    }
    const int run = sort_run(n, E);
    int32_t *hist = (int32_t *)((char *)ws + W4A16_WS_COUNTER_BYTES);
    hipLaunchKernelGGL(moe_sort_count_kernel, dim3(wgs), dim3(SORT_THREADS), 0, st, ids, n, run, E, hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_sort_place_kernel, dim3(wgs), dim3(SORT_THREADS), 0, st, ids, n, run, topk, E, bits, hist,
                       offsets, row_token, slot_row);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const void *Y, int dtype, const int32_t *slot_row,
                              const float *weights, int T, int topk, int M_rows, int N, void *out,
                              hipStream_t st)
{
    const bool wide = N % 8 == 0 && ((uintptr_t)Y & 15) == 0 && ((uintptr_t)out & 15) == 0;
    const bool bf = dtype == QG_DT_BF16;
    const int cols = wide ? N / 8 : N;
    // a grid's y extent holds 65535 tokens
    for (int t0 = 0; t0 < T; t0 += 65535) {
        const dim3 grid((cols + 255) / 256, T - t0 < 65535 ? T - t0 : 65535), block(256);
        const int32_t *row = slot_row + (size_t)t0 * topk;
        const float *w = weights + (size_t)t0 * topk;
        const uint16_t *y = (const uint16_t *)Y;
        uint16_t *o = (uint16_t *)out + (size_t)t0 * N;
#define QG_COMBINE(KERN, BF) hipLaunchKernelGGL((KERN<BF>), grid, block, 0, st, y, row, w, topk, M_rows, N, o)
        if (wide && bf) QG_COMBINE(moe_combine_kernel, true);
        else if (wide) QG_COMBINE(moe_combine_kernel, false);
        else if (bf) QG_COMBINE(moe_combine_narrow_kernel, true);
        else QG_COMBINE(moe_combine_narrow_kernel, false);
#undef QG_COMBINE
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

} // namespace qg
