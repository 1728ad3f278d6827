// Attention over the paged 4-bit cache (layout in qg_kv4.h): one pass over the
// tokens with the running maximum and sum of a softmax, on the fp16 MFMA.
//
// With K = kc ks + kz and V = vc vs + vz by token t and group g of channels,
//   score[t]  = sum_g ks[t,g] (q_g . kc[t]_g) + kz[t,g] sum(q_g)
//   out_g     = sum_t (p[t] vs[t,g]) vc[t]_g + sum_t p[t] vz[t,g]
// so the codes go into the products as they are (exact binary16 subnormals, two ANDs
// and a shift per four of them) and scales and zeros stay in 32 bits outside.  The
// only operands rounded to 16 bits are p[t] vs[t,g]; the queries enter exactly, scaled
// by a power of two of their row's largest value (bf16 ones too: eight bits of eleven).
//
// A wave takes 16 NQ rows (the query heads of one key/value head, token by token) as
// the columns of its products and the tokens as the rows: a lane then holds the scores of
// one query row against four consecutive tokens of each of two 16-token tiles, which
// is what the second product takes from it, and nothing goes through LDS.
#include "qg_kv4.h"
#include "qg_launch.h"

#include <type_traits>

namespace qg {
namespace {

struct AttendArgs {
    const uint16_t *q;
    uint16_t *out;
    long long ldq;
    int q_heads, R;                // R: query heads of one key/value head
    bool bf16;
    float scale;                   // softmax scale times log2 e
    int window, sinks;             // window 0: none
    int splits;                    // parts of a sequence's blocks
    float *part, *ml;              // [splits][T * q_heads][D] and [..][2], splits > 1
};

constexpr float NONE = -3.0e38f;   // the running maximum before any token
// A column's maximum is raised only when a score exceeds it by more than this power of
// two: p <= 4 and p * vs <= 4 * 8736 (a scale is at most 2 * 65504 / 15) stays a
// binary16, and the rescaling of all accumulators is rare.
constexpr float SLACK = 2.0f;

// The two k-steps of a word pair (K), or the operand of one word (V).
__device__ inline half8 code_op(unsigned x, unsigned y, unsigned mask)
{
    return __builtin_bit_cast(half8, uint4v{x & mask, x >> 8 & mask, y & mask, y >> 8 & mask});
}
__device__ inline half8 value_op(unsigned x)
{
    return __builtin_bit_cast(half8, uint4v{x & 0x000F000Fu, x >> 8 & 0x000F000Fu, x & 0x00F000F0u, x >> 8 & 0x00F000F0u});
}

__device__ inline float lo16(unsigned x) { return h2f((uint16_t)x); }
__device__ inline float hi16(unsigned x) { return h2f((uint16_t)(x >> 16)); }

template <int D, int NG>
struct Stage {
    static constexpr int NW = D / 32;
    unsigned k[2][NW];
    uint4v v[D / 64];
    uint4v ks[NG][2], vs[NG][2];
    int t0;
    bool ok;
};

// MERGE: the workgroup's four waves share 16 NQ rows and take every fourth block of
// tokens; their results meet in LDS at the end.  Otherwise each wave has rows of its own.
template <int D, int NG, int NQ, bool MERGE>
__global__ __launch_bounds__(256) void kv4_attend_kernel(Kv4Cache c, Kv4Batch s, AttendArgs a)
{
    constexpr int NW = D / 32, DT = D / 16, SPG = NW / NG, TPG = DT / NG;
    constexpr int ROWS = 16 * NQ, RB = MERGE ? ROWS : 4 * ROWS;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, kq = lane >> 4;
    const int H = c.heads, R = a.R;
    const int h = blockIdx.x % H, xs = blockIdx.x / H;
    const int split = xs % a.splits;
    int b, in, of;
    Run seq;
    if (!kv4_find(s, xs / a.splits, [=](const Run &q) { return (q.n * R + RB - 1) / RB; }, b, in, of, seq)) return;
    in = of - 1 - in;                                      // the longest first
    const int rows = seq.n * R;
    const int row0 = in * RB + (MERGE ? 0 : w * ROWS);
    if (row0 >= rows) return;
    const int last = row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1;
    const int first = seq.len - seq.n;                     // position of the first row's token
    const int p0 = first + row0 / R, p1 = first + last / R;

    // the blocks of tokens that any of the rows sees: the sinks', then the window's
    const int cap = s.width << c.shift;
    const int end = p1 < cap ? p1 : cap - 1;
    int ns = 0, w0 = 0, nb = 0;
    if (end >= 0) {
        if (a.window) {
            const int from = p0 - a.window + 1;
            w0 = from > 0 ? from >> 5 : 0;
            ns = (a.sinks + 31) >> 5;
            if (w0 > end >> 5) w0 = (end >> 5) + 1;
            ns = ns < w0 ? ns : w0;
        }
        nb = ns + (end >> 5) - w0 + 1;
    }
    int per = (nb + a.splits - 1) / a.splits;
    if (MERGE) per = (per + 3) & ~3;
    const int j0 = split * per, j1 = j0 + per < nb ? j0 + per : nb;
    const int step = MERGE ? 4 : 1;

    // the rows: operand, group sums, factor of their scores, position
    half8 qo[NQ][NW];
    float qs[NQ][NG], f[NQ];
    int pos[NQ];
    size_t grow[NQ];                                       // row of [T * q_heads]
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = row0 + 16 * n + col;
        const bool live = r < rows;
        const int i = live ? r / R : 0, hr = live ? r - i * R : 0;
        const size_t t = (size_t)seq.row + i;
        grow[n] = t * a.q_heads + (size_t)h * R + hr;
        pos[n] = live ? first + i : -1;
        const uint16_t *const p = a.q + t * a.ldq + ((size_t)h * R + hr) * D + 8 * kq;
        float x[NW][8], big = 0.0f;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const uint4v raw = *reinterpret_cast<const uint4v *>(p + 32 * k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint16_t v = (uint16_t)(raw[e >> 1] >> (16 * (e & 1)));
                x[k][e] = live ? (a.bf16 ? bf2f(v) : h2f(v)) : 0.0f;
                bad |= !(__builtin_fabsf(x[k][e]) < __builtin_inff());
                big = fmaxf(big, __builtin_fabsf(x[k][e]));
            }
        }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        bad |= __shfl_xor((int)bad, 16) != 0;
        bad |= __shfl_xor((int)bad, 32) != 0;
        int ex = 0;
        if (big > 0.0f && !bad) (void)frexpf(big, &ex);    // big < 2^ex
        // q' = q 2^(15 - ex), below 2^15; the codes weigh 2^-24
        f[n] = bad ? __builtin_nanf("") : ldexpf(a.scale, ex + 9);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float sum = 0.0f;
#pragma unroll
            for (int k = g * SPG; k < (g + 1) * SPG; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[k][e] = ldexpf(x[k][e], 15 - ex);
                    sum += x[k][e];
                    qo[n][k][e] = (_Float16)(k < NW / 2 ? x[k][e] : 0.0625f * x[k][e]);
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            qs[n][g] = sum * 0x1p-24f;
        }
    }

    float m[NQ], l[NQ][2], z[NQ][NG][2];
    float4v o[NQ][DT];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = NONE;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g) z[n][g][0] = z[n][g][1] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = float4v{0, 0, 0, 0};
    }

    auto load = [&](Stage<D, NG> &x, int j) {
        const int blk = j < ns ? j : j - ns + w0;
        x.t0 = blk << 5;
        const int pg = s.table[(size_t)b * s.width + (x.t0 >> c.shift)];
        x.ok = (unsigned)pg < (unsigned)c.pages;
        const size_t head = (size_t)(x.ok ? pg : 0) * H + h;
        const int tin = x.t0 & ((1 << c.shift) - 1);
        const size_t at = ((head << c.shift) + tin) * (D / 8);
        const uint32_t *const kp = c.k + at + col * (D / 8) + kq * NW;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (NW == 2) {
                const uint2v r = *reinterpret_cast<const uint2v *>(kp + t * 16 * (D / 8));
                x.k[t][0] = r.x;
                x.k[t][1] = r.y;
            } else {
#pragma unroll
                for (int i = 0; i < NW / 4; ++i) {
                    const uint4v r = *reinterpret_cast<const uint4v *>(kp + t * 16 * (D / 8) + 4 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x.k[t][4 * i + e] = r[e];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            x.v[u] = *reinterpret_cast<const uint4v *>(c.v + at + u * 256 + lane * 4);
        const size_t sat = ((head * NG) << c.shift) + tin + 4 * kq;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                x.ks[g][t] = *reinterpret_cast<const uint4v *>(c.k_sz + sat + ((size_t)g << c.shift) + 16 * t);
                x.vs[g][t] = *reinterpret_cast<const uint4v *>(c.v_sz + sat + ((size_t)g << c.shift) + 16 * t);
            }
    };

    auto compute = [&](const Stage<D, NG> &x, auto masked) {
        constexpr bool MASK = decltype(masked)::value;
        float4v sc[NQ][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            half8 op[NW];
#pragma unroll
            for (int i = 0; i < NW / 2; ++i) {
                op[i] = code_op(x.k[t][2 * i], x.k[t][2 * i + 1], 0x000F000Fu);
                op[i + NW / 2] = code_op(x.k[t][2 * i], x.k[t][2 * i + 1], 0x00F000F0u);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    float4v acc = {0, 0, 0, 0};
#pragma unroll
                    for (int k = g * SPG; k < (g + 1) * SPG; ++k) acc = mfma_f16(op[k], qo[n][k], acc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float zero = hi16(x.ks[g][t][r]) * qs[n][g];
                        sc[n][t][r] = lo16(x.ks[g][t][r]) * acc[r] + (g ? sc[n][t][r] + zero : zero);
                    }
                }
        }
        bool vis[NQ][2][4];
        if (MASK) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = x.t0 + 16 * t + 4 * kq + r;
                        vis[n][t][r] = x.ok && at <= pos[n] &&
                                       (!a.window || at > pos[n] - a.window || at < a.sinks);
                        if (!vis[n][t][r]) sc[n][t][r] = -__builtin_inff();
                    }
        }
        bool raise = false;
        float mx[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float v = fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3]));
            v = fmaxf(v, fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3])));
            mx[n] = v * f[n];                              // (f > 0)
            raise |= mx[n] > m[n] + SLACK;
        }
        if (__any(raise)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float v = fmaxf(mx[n], __shfl_xor(mx[n], 16));
                v = fmaxf(m[n], fmaxf(v, __shfl_xor(v, 32)));
                const float by = __builtin_amdgcn_exp2f(m[n] - v);
                m[n] = v;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    l[n][t] *= by;
#pragma unroll
                    for (int g = 0; g < NG; ++g) z[n][g][t] *= by;
                }
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] *= by;
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // the second tile's codes are the high nibbles: 16 times as large
                    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][t][r], f[n], -(m[n] + (t ? 4.0f : 0.0f))));
                    sc[n][t][r] = MASK && !vis[n][t][r] ? 0.0f : p;
                    l[n][t] += sc[n][t][r];
                }
        half8 vo[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) vo[d] = value_op(x.v[d / 4][d % 4]);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                half8 po;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float vs = lo16(x.vs[g][t][r]), vz = hi16(x.vs[g][t][r]);
                        if (MASK) {
                            vs = vis[n][t][r] ? vs : 0.0f;
                            vz = vis[n][t][r] ? vz : 0.0f;
                        }
                        po[4 * t + r] = (_Float16)(sc[n][t][r] * vs);
                        z[n][g][t] = __builtin_fmaf(sc[n][t][r], vz, z[n][g][t]);
                    }
#pragma unroll
                for (int d = g * TPG; d < (g + 1) * TPG; ++d) o[n][d] = mfma_f16(vo[d], po, o[n][d]);
            }
    };

    auto block = [&](const Stage<D, NG> &x) {
        debug_stage_sync();
        // all rows see all of the block, or some do not
        const bool whole = x.ok && x.t0 + 31 <= p0 &&
                           (!a.window || x.t0 > p1 - a.window || x.t0 + 31 < a.sinks);
        if (whole)
            compute(x, std::false_type{});
        else
            compute(x, std::true_type{});
    };

    for (int j = j0 + (MERGE ? w : 0); j < j1; j += step) {
        Stage<D, NG> x;
        load(x, j);
        block(x);
    }

    // a column's sums over its four lanes, and its values with the zeros' part
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        float sum = l[n][0] + 16.0f * l[n][1];
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        l[n][0] = sum;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float zs = z[n][g][0] + 16.0f * z[n][g][1];
            zs += __shfl_xor(zs, 16);
            zs += __shfl_xor(zs, 32);
#pragma unroll
            for (int d = g * TPG; d < (g + 1) * TPG; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[n][d][r] = __builtin_fmaf(o[n][d][r], 0x1p24f, zs);
        }
    }

    const size_t all = (size_t)s.T * a.q_heads;
    if constexpr (MERGE) {
        constexpr int LD = D + 4;
        __shared__ float so[4][16][LD];
        __shared__ float sm[4][16], sl[4][16];
        // what a thread adds up: four channels of a row
        constexpr int TPR = D / 4, PASS = 256 / TPR;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            if (n) __syncthreads();
#pragma unroll
            for (int d = 0; d < DT; ++d)
                *reinterpret_cast<float4v *>(&so[w][col][16 * d + 4 * kq]) = o[n][d];
            if (kq == 0) {
                sm[w][col] = m[n];
                sl[w][col] = l[n][0];
            }
            debug_stage_sync();
            __syncthreads();
            for (int r = threadIdx.x / TPR; r < 16 && row0 + 16 * n + r < rows; r += PASS) {
                const int ch = threadIdx.x % TPR * 4;
                const float mm = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
                float sum = 0.0f;
                float4v acc = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float by = __builtin_amdgcn_exp2f(sm[i][r] - mm);
                    sum += by * sl[i][r];
                    acc += by * *reinterpret_cast<const float4v *>(&so[i][r][ch]);
                }
                const int rr = row0 + 16 * n + r, i = rr / R;
                const size_t g = ((size_t)seq.row + i) * a.q_heads + (size_t)h * R + (rr - i * R);
                if (a.splits > 1) {
                    if (ch == 0) {
                        a.ml[(split * all + g) * 2] = mm;
                        a.ml[(split * all + g) * 2 + 1] = sum;
                    }
                    if (j0 < j1) *reinterpret_cast<float4v *>(a.part + (split * all + g) * D + ch) = acc;
                } else {
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    uint2v r2;
                    uint16_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = a.bf16 ? f2bf(acc[e] * inv) : f2h(acc[e] * inv);
                    r2.x = v[0] | (uint32_t)v[1] << 16;
                    r2.y = v[2] | (uint32_t)v[3] << 16;
                    *reinterpret_cast<uint2v *>(a.out + g * D + ch) = r2;
                }
            }
        }
    } else {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            if (row0 + 16 * n + col >= rows) continue;
            if (a.splits > 1) {
                if (kq == 0) {
                    a.ml[(split * all + grow[n]) * 2] = m[n];
                    a.ml[(split * all + grow[n]) * 2 + 1] = l[n][0];
                }
                if (j0 < j1)
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        *reinterpret_cast<float4v *>(a.part + (split * all + grow[n]) * D + 16 * d + 4 * kq) = o[n][d];
                continue;
            }
            const float inv = l[n][0] == 0.0f ? 0.0f : 1.0f / l[n][0];
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                uint16_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = a.bf16 ? f2bf(o[n][d][e] * inv) : f2h(o[n][d][e] * inv);
                *reinterpret_cast<uint2v *>(a.out + grow[n] * D + 16 * d + 4 * kq) =
                    uint2v{v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16};
            }
        }
    }
}

// The parts of a row, one workgroup a row: groups of D / 4 threads take every further
// part, then meet in LDS.  Parts without a token hold sum 0 and no values.
template <int D>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4Batch s, AttendArgs a)
{
    constexpr int TPR = D / 4, GR = 256 / TPR;
    const size_t all = (size_t)s.T * a.q_heads, g = blockIdx.x;
    if (s.off) {                                          // rows of no sequence stay as they are
        const long long t = (long long)(g / a.q_heads);
        if (t < s.off[0] || t >= s.off[s.B]) return;
    }
    const int grp = threadIdx.x / TPR, ch = threadIdx.x % TPR * 4;
    float m = NONE;
    for (int i = 0; i < a.splits; ++i) m = fmaxf(m, a.ml[(i * all + g) * 2]);
    float sum = 0.0f;
    float4v acc = {0, 0, 0, 0};
    for (int i = grp; i < a.splits; i += GR) {
        const float mi = a.ml[(i * all + g) * 2], li = a.ml[(i * all + g) * 2 + 1];
        if (li == 0.0f) continue;
        const float by = __builtin_amdgcn_exp2f(mi - m);
        sum += by * li;
        acc += by * *reinterpret_cast<const float4v *>(a.part + (i * all + g) * D + ch);
    }
    __shared__ float4v so[GR][TPR];
    __shared__ float sl[GR];
    so[grp][threadIdx.x % TPR] = acc;
    if (ch == 0) sl[grp] = sum;
    debug_stage_sync();
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 1; i < GR; ++i) {
        acc += so[i][threadIdx.x];
        sum += sl[i];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = a.bf16 ? f2bf(acc[e] * inv) : f2h(acc[e] * inv);
    *reinterpret_cast<uint2v *>(a.out + g * D + ch) = uint2v{v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16};
}

template <int D, int NG>
void launch_attend(const Kv4AttendPlan &p, const Kv4Cache &c, const Kv4Batch &s, const AttendArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)p.workgroups);
    if (p.shared)
        hipLaunchKernelGGL((kv4_attend_kernel<D, NG, 1, true>), grid, dim3(256), 0, st, c, s, a);
    else
        hipLaunchKernelGGL((kv4_attend_kernel<D, NG, D == 256 ? 1 : 2, false>), grid, dim3(256), 0, st, c, s, a);
}

} // namespace

// Decode batches (up to 16 rows of a key/value head in a sequence): the four waves of
// a workgroup share the rows.  More rows: each wave has 32 of its own (16 of 256 channels).
Kv4AttendPlan kv4_attend_plan(int T, int max_new, int B, int q_heads, int heads, int D, int max_tokens, int window,
                              int sinks)
{
    Kv4AttendPlan p;
    const long long R = q_heads / heads;
    p.shared = max_new * R <= 16;
    p.rows = p.shared || D == 256 ? 16 : 32;
    const int rb = p.shared ? p.rows : 4 * p.rows;
    // row blocks of all sequences: each has at most one that is not full
    const long long blocks = T * R / rb + (T < B ? T : B);
    long long tokens = max_tokens;
    if (window > 0) {
        const long long seen = (long long)window + sinks + max_new + 64;
        tokens = seen < tokens ? seen : tokens;
    }
    const long long most = (tokens + 127) / 128;          // four blocks of tokens to a part
    long long n = (1024 + blocks * heads - 1) / (blocks * heads);
    n = n > most ? most : n;
    n = n > 128 ? 128 : n;
    p.splits = n < 1 ? 1 : (int)n;
    p.workgroups = blocks * heads * p.splits;
    p.bytes = p.splits == 1 ? 0 : (size_t)p.splits * T * q_heads * (D + 2) * sizeof(float);
    return p;
}

hipError_t launch_kv4_attend(const Kv4AttendPlan &p, const Kv4Cache &c, const Kv4Batch &s, const void *q, long long ldq,
                             int q_heads, int dtype, float scale, int window, int sinks, void *out, void *ws,
                             hipStream_t st)
{
    const size_t all = (size_t)s.T * q_heads;
    float *const part = (float *)ws;
    const AttendArgs a = {(const uint16_t *)q, (uint16_t *)out, ldq, q_heads, q_heads / c.heads, dtype == QG_DT_BF16,
                          scale * 1.4426950408889634f, window, sinks, p.splits, part,
                          part ? part + (size_t)p.splits * all * c.D : nullptr};
    const int ng = c.D / c.g;
#define QG_ATTEND(DIM, GROUPS) \
    if (c.D == DIM && ng == GROUPS) launch_attend<DIM, GROUPS>(p, c, s, a, st)
    QG_ATTEND(64, 1);
    else QG_ATTEND(64, 2);
    else QG_ATTEND(128, 1);
    else QG_ATTEND(128, 2);
    else QG_ATTEND(128, 4);
    else QG_ATTEND(256, 2);
    else QG_ATTEND(256, 4);
    else QG_ATTEND(256, 8);
    else return hipErrorInvalidValue;
#undef QG_ATTEND
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    switch (c.D) {
    case 64: hipLaunchKernelGGL((kv4_join_kernel<64>), dim3((unsigned)all), dim3(256), 0, st, s, a); break;
    case 128: hipLaunchKernelGGL((kv4_join_kernel<128>), dim3((unsigned)all), dim3(256), 0, st, s, a); break;
    default: hipLaunchKernelGGL((kv4_join_kernel<256>), dim3((unsigned)all), dim3(256), 0, st, s, a); break;
    }
    return hipGetLastError();
}

} // namespace qg
