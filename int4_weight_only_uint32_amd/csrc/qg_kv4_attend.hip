// Attention over the paged 4-bit cache (layout in qg_kv4.h): one pass over the
// tokens with the running maximum and sum of a softmax, on the fp16 MFMA.
//
// With K = kc ks + kz and V = vc vs + vz by token t and group g of channels,
//   score[t]  = sum_g ks[t,g] (q_g . kc[t]_g) + kz[t,g] sum(q_g)
//   out_g     = sum_t (p[t] vs[t,g]) (vc[t]_g - 8) + sum_t p[t] (vz[t,g] + 8 vs[t,g])
// so codes enter the products exactly: keys as the binary16 subnormals that an AND
// leaves of their nibbles (two ANDs and half a shift for two of them), values, whose
// partner p vs is rounded to 16 bits, around their middle, where that rounding costs a
// third of what it would around 0 (a packed subtraction more).  The terms of the zeros
// are one more product each, straight from the words in which scale and zero stand: for the
// keys against sum(q_g) as two 16-bit values, for the values against p, together with
// a row of ones that sums p up.  The queries enter exactly, scaled by a power of two of
// their row's largest value (bf16 ones too: eight bits of eleven).
//
// A wave takes 16 NQ rows (the query heads of one key/value head, token by token) as
// the columns of its products and the tokens as the rows: a lane then holds the scores of
// one query row against four consecutive tokens of each of two 16-token tiles, which
// is what the second product takes from it.
#include "qg_kv4.h"
#include "qg_launch.h"

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

// A k-step of a pair of key words: their low (high) nibbles, 2^-24 (2^-20) each.
__device__ inline half8 code_op(unsigned x, unsigned y, unsigned mask)
{
    return __builtin_bit_cast(half8, uint4v{x & mask, x >> 8 & mask, y & mask, y >> 8 & mask});
}
// The eight codes of a value word, less 8: a low nibble ORed into 0x6400 reads 1024 + v, a
// high one into 0x5400 64 + v, and the subtraction is exact.
__device__ inline half8 value_op(unsigned x, unsigned mag_lo, unsigned mag_hi)
{
    const half2v off_lo = {(_Float16)1032.f, (_Float16)1032.f}, off_hi = {(_Float16)72.f, (_Float16)72.f};
    const unsigned y = x >> 8;
    auto lo = [&](unsigned v) {
        return __builtin_bit_cast(unsigned, __builtin_bit_cast(half2v, and_or_b32(v, 0x000F000Fu, mag_lo)) - off_lo);
    };
    auto hi = [&](unsigned v) {
        return __builtin_bit_cast(unsigned, __builtin_bit_cast(half2v, and_or_b32(v, 0x00F000F0u, mag_hi)) - off_hi);
    };
    return __builtin_bit_cast(half8, uint4v{lo(x), lo(y), hi(x), hi(y)});
}

// Whether either half of a word is no finite binary16.
__device__ inline bool odd_word(unsigned w)
{
    return (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
}

__device__ inline float lo16(unsigned x) { return h2f((uint16_t)x); }

template <int N>
__device__ inline void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A wave's ring of 32-token blocks in LDS.  Loads go there directly: keys and values
// as they lie, then scales and zeros, [keys | values][group][32] words (repeated up
// to whole loads of 64 lanes).
template <int D, int NG>
struct Ring {
    static constexpr int STAGES = 2;
    static constexpr int CODES = 32 * D / 2;                       // bytes of a block's keys, or of its values
    static constexpr int SCALES = NG > 4 ? 256 * NG : 1024;
    static constexpr int BYTES = 2 * CODES + SCALES;
    static constexpr int LOADS = BYTES / 1024;
};

// MERGE: the workgroup's four waves share 16 NQ rows and take every fourth block of
// tokens; their results meet in LDS at the end.  Otherwise each wave has rows of its own.
template <int D, int NG, int NQ, bool MERGE>
__global__ __launch_bounds__(256, MERGE && D < 256 ? 3 : 2) void kv4_attend_kernel(Kv4Cache c, Kv4Batch s, AttendArgs a)
{
    constexpr int NW = D / 32, DT = D / 16, SPG = NW / NG, TPG = DT / NG;
    constexpr int ROWS = 16 * NQ, RB = MERGE ? ROWS : 4 * ROWS;
    using RG = Ring<D, NG>;
    constexpr int LD = D + 4;                              // (a row of the waves' results)
    constexpr int RINGS = 4 * RG::STAGES * RG::BYTES, SUMS = MERGE ? 4 * 16 * (LD + 2) * 4 : 0;
    // (one array for all: with several the compiler puts a wait for all loads before each
    // read of the ring)
    __shared__ __attribute__((aligned(16))) uint8_t lds[RINGS > SUMS ? RINGS : SUMS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, kq = lane >> 4;
    const int H = c.heads, R = a.R;
    uint8_t *const ring = lds + w * (RG::STAGES * RG::BYTES);
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

    // the rows' queries, and positions
    uint4v raw[NQ][NW];
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
#pragma unroll
        for (int k = 0; k < NW; ++k) raw[n][k] = *reinterpret_cast<const uint4v *>(p + 32 * k);
    }

    // a wave's blocks: every `step`-th from j0 + (its number) on
    const int mine = j1 <= j0 ? 0 : (MERGE ? (j1 - j0 - w + 3) / 4 : j1 - j0);
    auto block_of = [&](int i) {
        const int j = j0 + (MERGE ? w : 0) + i * step;
        return j < ns ? j : j - ns + w0;
    };
    auto page_of = [&](int i) { return s.table[(size_t)b * s.width + (block_of(i) >> (c.shift - 5))]; };
    constexpr int SLOADS = RG::SCALES / 1024;
    const uint32_t *sz0[SLOADS];
#pragma unroll
    for (int u = 0; u < SLOADS; ++u) {
        const int piece = (8 * u + lane / 8) % (2 * NG);
        sz0[u] = (piece < NG ? c.k_sz : c.v_sz) + ((size_t)(piece % NG) << c.shift) + lane % 8 * 4;
    }
    auto load = [&](int i, int pg) {
        const int t0 = block_of(i) << 5, tin = t0 & ((1 << c.shift) - 1);
        const size_t head = (size_t)((unsigned)pg < (unsigned)c.pages ? pg : 0) * H + h;
        const size_t at = ((head << c.shift) + tin) * (D / 8);
        uint8_t *const to = ring + (i % RG::STAGES) * RG::BYTES;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) lds_load16<0>(c.k + at + u * 256 + lane * 4, to + u * 1024);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) lds_load16<0>(c.v + at + u * 256 + lane * 4, to + RG::CODES + u * 1024);
        const size_t sat = ((head * NG) << c.shift) + tin;
#pragma unroll
        for (int u = 0; u < SLOADS; ++u) lds_load16<0>(sz0[u] + sat, to + 2 * RG::CODES + u * 1024);
    };

    // pages are asked for two blocks ahead, blocks one
    int pg = 0, next = 0;
    if (mine > 0) {
        pg = page_of(0);
        next = page_of(mine > 1 ? 1 : 0);
        load(0, pg);
    }

    // the queries as operands, q' = q 2^(15 - ex) below 2^15 (sixteenths against the high
    // nibbles); the factor of the scores (the codes weigh 2^-24); the groups' sums as two
    // 16-bit values, against the zeros in the words of lane groups 0 (the upper part) and 1
    half8 qo[NQ][NW], qz[NQ];
    float f[NQ];
    constexpr int GL = NG > 4 ? 2 : 1;                     // lane groups that the groups' words take
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        float x[NW][8], big = 0.0f;
        bool bad = false;
        const bool live = pos[n] >= 0 || row0 + 16 * n + col < rows;
#pragma unroll
        for (int k = 0; k < NW; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint16_t v = live ? (uint16_t)(raw[n][k][e >> 1] >> (16 * (e & 1))) : 0;
                const float fb = bf2f(v), fh = h2f(v);
                x[k][e] = a.bf16 ? fb : fh;
                bad |= !(__builtin_fabsf(x[k][e]) < __builtin_inff());
                big = fmaxf(big, __builtin_fabsf(x[k][e]));
            }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        bad |= __shfl_xor((int)bad, 16) != 0;
        bad |= __shfl_xor((int)bad, 32) != 0;
        int ex = 0;
        if (big > 0.0f && !bad) (void)frexpf(big, &ex);    // big < 2^ex
        f[n] = bad ? __builtin_nanf("") : ldexpf(a.scale, ex + 9);
        float qs[NG];
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
            qs[g] = sum * 0x1p-24f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = 0.0f;
            if (NG > 4)
                v = (kq & 1) ? qs[(4 + i) % NG] : qs[i % NG];
            else if (i < NG)
                v = qs[i];
            const _Float16 hi = (_Float16)v;
            const _Float16 part = kq / GL == 0 ? hi : kq / GL == 1 ? (_Float16)(v - (float)hi) : (_Float16)0.0f;
            qz[n][2 * i] = (_Float16)0.0f;
            qz[n][2 * i + 1] = part;
        }
    }

    // running maximum; products with the values' codes; with their scales (even rows) and
    // zeros (odd), and with ones (row 2 NG: the sum of p; with eight groups no row is left)
    constexpr bool LROW = 2 * NG < 16;
    float m[NQ], l[NQ];
    float4v o[NQ][DT], z[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        m[n] = NONE;
        l[n] = 0.0f;
        z[n] = float4v{0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = float4v{0, 0, 0, 0};
    }
    unsigned mag_lo = 0x64006400u, mag_hi = 0x54005400u;
    pin(mag_lo);
    pin(mag_hi);

    auto block = [&](const uint8_t *x, int t0, bool ok) {
        const uint4v *const ksz = reinterpret_cast<const uint4v *>(x + 2 * RG::CODES) + kq;
        const uint4v *const vsz = ksz + NG * 8;
        const unsigned *const kw = reinterpret_cast<const unsigned *>(x + 2 * RG::CODES) + col;
        float4v sc[NQ][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            half8 op[NW];
            const uint8_t *const kt = x + t * (RG::CODES / 2) + (col * 4 + kq) * (D / 8);
#pragma unroll
            for (int i = 0; i < NW / 2; i += 2) {
                uint4v r = {0, 0, 0, 0};
                if constexpr (NW == 2) {
                    const uint2v r2 = *reinterpret_cast<const uint2v *>(kt);
                    r.x = r2.x;
                    r.y = r2.y;
                } else {
                    r = *reinterpret_cast<const uint4v *>(kt + 8 * i);
                }
                op[i] = code_op(r.x, r.y, 0x000F000Fu);
                op[i + NW / 2] = code_op(r.x, r.y, 0x00F000F0u);
                if constexpr (NW > 2) {
                    op[i + 1] = code_op(r.z, r.w, 0x000F000Fu);
                    op[i + 1 + NW / 2] = code_op(r.z, r.w, 0x00F000F0u);
                }
            }
            uint4v zw = {0, 0, 0, 0};                      // this lane's token: (scale, zero) of four groups
#pragma unroll
            for (int i = 0; i < (NG < 4 ? NG : 4); ++i)
                zw[i] = kw[(NG > 4 ? (kq & 1) * 4 + i : i) * 32 + 16 * t];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                sc[n][t] = mfma_f16(__builtin_bit_cast(half8, zw), qz[n], float4v{0, 0, 0, 0});
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint4v sz = ksz[g * 8 + t * 4];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    float4v acc = {0, 0, 0, 0};
#pragma unroll
                    for (int k = g * SPG; k < (g + 1) * SPG; ++k) acc = mfma_f16(op[k], qo[n][k], acc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[n][t][r] = __builtin_fmaf(lo16(sz[r]), acc[r], sc[n][t][r]);
                }
            }
        }
        // all rows see all of the block, or some do not: a bit for each score that is hidden
        const bool whole = ok && t0 + 31 <= p0 && (!a.window || t0 > p1 - a.window || t0 + 31 < a.sinks);
        unsigned hide[NQ];
        if (!whole) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                hide[n] = 0;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = t0 + 16 * t + 4 * kq + r;
                        const bool vis = ok && at <= pos[n] && (!a.window || at > pos[n] - a.window || at < a.sinks);
                        hide[n] |= vis ? 0u : 1u << (4 * t + r);
                        sc[n][t][r] = vis ? sc[n][t][r] : -__builtin_inff();
                    }
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
                l[n] *= by;
                z[n] *= by;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[n][d] *= by;
            }
        }
        half8 pf[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sc[n][t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][t][r], f[n], -m[n]));
        if (!whole) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (hide[n] >> (4 * t + r) & 1) sc[n][t][r] = 0.0f;
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    pf[n][4 * t + r] = (_Float16)sc[n][t][r];
                    if (!LROW) l[n] += sc[n][t][r];
                }

        // the rows of scales and zeros: lane (col, kq) takes the halves of one kind of group
        // col / 2, of the eight tokens of lane group kq
        const int zg = col / 2 < NG ? col / 2 : 0;
        uint4v za[2], zh;
#pragma unroll
        for (int t = 0; t < 2; ++t) za[t] = vsz[zg * 8 + t * 4];
        if (!whole) {
            // a token that one row sees and another does not must not bring it a NaN: 0 here, and a NaN
            // put in where it is seen
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) za[t][r] = odd_word(za[t][r]) ? 0u : za[t][r];
        }
        const unsigned sel = (col & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            zh[2 * t] = __builtin_amdgcn_perm(za[t][1], za[t][0], sel);
            zh[2 * t + 1] = __builtin_amdgcn_perm(za[t][3], za[t][2], sel);
        }
        if (LROW && col >= 2 * NG) zh = uint4v{0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
#pragma unroll
        for (int n = 0; n < NQ; ++n) z[n] = mfma_f16(__builtin_bit_cast(half8, zh), pf[n], z[n]);

#pragma unroll
        for (int g = 0; g < NG; ++g) {
            uint4v sz[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) sz[t] = vsz[g * 8 + t * 4];
            if (!whole) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    bool nan = false;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) nan |= odd_word(sz[t][r]) && !(hide[n] >> (4 * t + r) & 1);
                    if (__any(nan)) {
                        int any = nan;
                        any |= __shfl_xor(any, 16);
                        any |= __shfl_xor(any, 32);
                        if (any && kq == g / 2) z[n][2 * (g % 2)] = __builtin_nanf("");
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sz[t][r] = odd_word(sz[t][r]) ? 0u : sz[t][r];
            }
            half8 po[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) po[n][4 * t + r] = (_Float16)__builtin_fmaf(lo16(sz[t][r]), sc[n][t][r], 0.0f);
#pragma unroll
            for (int d = g * TPG; d < (g + 1) * TPG; ++d) {
                const half8 vo = value_op(*reinterpret_cast<const unsigned *>(x + RG::CODES + d / 4 * 1024 + lane * 16 + d % 4 * 4),
                                          mag_lo, mag_hi);
#pragma unroll
                for (int n = 0; n < NQ; ++n) o[n][d] = mfma_f16(vo, po[n], o[n][d]);
            }
        }
    };

    for (int i = 0; i < mine; ++i) {
        const int here = pg;
        pg = next;
        if (i + 1 < mine) {
            next = page_of(i + 2 < mine ? i + 2 : i + 1);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage's last reads are done
            load(i + 1, pg);
            debug_stage_sync();
            wait_loads<RG::LOADS>();
        } else {
            wait_loads<0>();
        }
        block(ring + (i % RG::STAGES) * RG::BYTES, block_of(i) << 5, (unsigned)here < (unsigned)c.pages);
    }

    // a column's sum of p, and its values with the zeros' part, from the lane groups that hold them
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        if (LROW) {
            l[n] = __shfl(z[n][2 * NG % 4], 16 * (2 * NG / 4 % 4) + col);
        } else {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
        }
        const float zz[2] = {__builtin_fmaf(z[n][0], 8.0f, z[n][1]), __builtin_fmaf(z[n][2], 8.0f, z[n][3])};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float zs = __shfl(zz[g % 2], 16 * (g / 2) + col);
#pragma unroll
            for (int d = g * TPG; d < (g + 1) * TPG; ++d) o[n][d] += zs;
        }
    }

    const size_t all = (size_t)s.T * a.q_heads;
    if constexpr (MERGE) {
        float(*const so)[16][LD] = reinterpret_cast<float(*)[16][LD]>(lds);
        float(*const sm)[16] = reinterpret_cast<float(*)[16]>(lds + 4 * 16 * LD * 4), (*const sl)[16] = sm + 4;
        __syncthreads();                                   // (the waves' rings are done with)
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
                sl[w][col] = l[n];
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
                    a.ml[(split * all + grow[n]) * 2 + 1] = l[n];
                }
                if (j0 < j1)
#pragma unroll
                    for (int d = 0; d < DT; ++d)
                        *reinterpret_cast<float4v *>(a.part + (split * all + grow[n]) * D + 16 * d + 4 * kq) = o[n][d];
                continue;
            }
            const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
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

// The parts of a row, one workgroup a row: a thread takes a part's maximum and sum, then
// groups of D / 4 threads every further part's values, and they meet in LDS.  Parts
// without a token hold sum 0 and no values.
constexpr int MAX_SPLITS = 128;
template <int D>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4Batch s, AttendArgs a)
{
    constexpr int TPR = D / 4, GR = 256 / TPR;
    const size_t all = (size_t)s.T * a.q_heads, g = blockIdx.x;
    if (s.off) {                                          // rows of no sequence stay as they are
        const long long t = (long long)(g / a.q_heads);
        if (t < s.off[0] || t >= s.off[s.B]) return;
    }
    const int tid = threadIdx.x, grp = tid / TPR, ch = tid % TPR * 4;
    __shared__ float4v so[GR][TPR];
    __shared__ float by[MAX_SPLITS], top[2], total[2];
    // (two waves hold the parts)
    float mi = NONE, li = 0.0f;
    if (tid < a.splits) {
        mi = a.ml[(tid * all + g) * 2];
        li = a.ml[(tid * all + g) * 2 + 1];
    }
    float m = mi;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (tid < MAX_SPLITS && tid % 64 == 0) top[tid / 64] = m;
    debug_stage_sync();
    __syncthreads();
    m = fmaxf(top[0], top[1]);
    if (tid < MAX_SPLITS) {
        const float e = __builtin_amdgcn_exp2f(mi - m);
        // a part without a token has no values to be read
        by[tid] = li == 0.0f ? 0.0f : e;
        li = li == 0.0f ? 0.0f : li * e;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) li += __shfl_xor(li, o);
        if (tid % 64 == 0) total[tid / 64] = li;
    }
    debug_stage_sync();
    __syncthreads();
    float4v acc = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = grp; i < a.splits; i += GR) {
        const float e = by[i];
        if (e != 0.0f) acc += e * *reinterpret_cast<const float4v *>(a.part + (i * all + g) * D + ch);
    }
    so[grp][tid % TPR] = acc;
    debug_stage_sync();
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 1; i < GR; ++i) acc += so[i][tid];
    const float sum = total[0] + total[1];
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
    // row blocks of all sequences: each has at most one that is not full.  (The grid holds
    // them whatever max_new says; where it says that a sequence has one at most, parts are
    // made for that many.)
    const long long some = T < B ? T : B;
    const long long blocks = T * R / rb + some;
    const long long likely = (max_new * R <= rb ? some : blocks) * heads;
    long long tokens = max_tokens;
    if (window > 0) {
        const long long seen = (long long)window + sinks + max_new + 64;
        tokens = seen < tokens ? seen : tokens;
    }
    // parts along the tokens fill the CUs once (three workgroups each of 64 or 128 shared
    // channels, else two), of at least a block of tokens for each wave
    const long long most = (tokens + 127) / 128, fit = p.shared && D < 256 ? 768 : 512;
    long long n = fit / likely;
    n = n > most ? most : n;
    n = n > MAX_SPLITS ? MAX_SPLITS : n;
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
