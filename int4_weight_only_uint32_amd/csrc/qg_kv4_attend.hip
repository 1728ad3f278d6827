// Attention over the paged 4-bit cache (layout in qg_kv4.h): one pass over the
// tokens with the running maximum and sum of a softmax, on the fp16 MFMA.
//
// With K = kc ks + kz and V = vc vs + vz by token t and group g of channels,
//   score[t]  = sum_g ks[t,g] (q_g . kc[t]_g) + kz[t,g] sum(q_g)
//   out_g     = sum_t (p[t] vs[t,g]) (vc[t]_g - 8) + sum_t p[t] (vz[t,g] + 8 vs[t,g])
// Codes enter the products exactly, as 64 + code, and 64 times their other operand's sum is taken
// off again.  p vs is rounded to 16 bits; around the middle of the codes that costs a third
// of what it would around 0, so 8 times the sum of the rounded values is taken off, too (one
// product with ones for a group).  The terms of the zeros are one more product each, straight
// from the words in which scale and zero stand: for the keys against sum(q_g) as two 16-bit
// values, with the scales against -64 of it, for the values against p, together with
// a row of ones that sums p up.  The queries enter scaled by a power of two of
// their row's largest value, and so exactly down to 2^-17 of it (2^-28 of it below).
//
// A wave takes 16 NQ rows (the query heads of one key/value head, token by token) as
// the columns of its products and the tokens as the rows: a lane then holds the scores of
// one query row against four consecutive tokens of each of two 16-token tiles, which
// is what the second product takes from it.
#include <cmath>

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
    float scale;                   // softmax scale times log2 e, as scale 2^scale_ex
    int scale_ex;
    int window, sinks;             // window 0: none
    int splits, items;             // most parts of a row's blocks; items of all sequences (SHARED)
    float *part, *ml;              // splits > 1: [splits][T * q_heads][D], and [..][2] maxima and sums
    int32_t *parts;                // [T * q_heads]: how many of them
};

constexpr float NONE = -3.0e38f;   // the reference before any token
// A column's p are powers of two over a reference that lies `room` under a maximum of its
// scores, so that small p, and p times the scale of small values, are not lost to the
// binary16's subnormals.  The reference is raised only when a score exceeds that maximum by
// more than SLACK, so that rescaling all accumulators is rare.  p <= 2^(room + SLACK)
// stays a binary16, and so does p * vs for scales up to 2^(13 - room); larger ones take room
// away, down to -3 for the largest that there are.
constexpr float SLACK = 2.0f;
constexpr int ROOM = 13;

// Codes as operands, 64 + code: the nibble at the exponent of 64, in bits 4 to 7 of a half.  (Left
// as the subnormals that a mask alone makes of them, or as 1024 + code from bits 0 to 3, they
// would cost a third fewer instructions; but a product's sums are cut off at 2^-24 or so of its operands'
// exponents, and a subnormal's is that of 2^-14: measured up to 2^-12 of a code, always to
// one side, against 2^-16 of this form.)
constexpr float OFFSET = 64.0f;
// (no inline assembly: it would not keep the distance to a matrix instruction that reads its result)
__device__ inline unsigned codes2(unsigned x, unsigned sixty_four) { return (x & 0x00F000F0u) | sixty_four; }
// a k-step of a pair of key words, of their low or high nibbles
__device__ inline half8 key_op(unsigned x, unsigned y, bool high, unsigned sixty_four)
{
    const auto two = [=](unsigned v) { return codes2(v, sixty_four); };
    return high ? __builtin_bit_cast(half8, uint4v{two(x), two(x >> 8), two(y), two(y >> 8)})
                : __builtin_bit_cast(half8, uint4v{two(x << 4), two(x >> 4), two(y << 4), two(y >> 4)});
}
// the eight tokens of a value word, four of each tile
__device__ inline half8 value_op(unsigned x, unsigned sixty_four)
{
    const auto two = [=](unsigned v) { return codes2(v, sixty_four); };
    return __builtin_bit_cast(half8, uint4v{two(x << 4), two(x >> 4), two(x), two(x >> 8)});
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

// A wave's ring of two 32-token blocks in LDS.  Loads go there directly: keys and values
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

// The blocks of tokens that any row at positions p0 .. p1 sees: first the sinks' (0 .. ns - 1), then
// the window's (from w0 on), nb in all.
struct SeenBlocks {
    int ns, w0, nb;
};
__device__ inline SeenBlocks seen_blocks(int p0, int p1, int window, int sinks, int cap)
{
    SeenBlocks r = {0, 0, 0};
    const int end = p1 < cap ? p1 : cap - 1;
    if (end < 0) return r;
    if (window) {
        const int from = p0 - window + 1;
        r.w0 = from > 0 ? from >> 5 : 0;
        if (r.w0 > end >> 5) r.w0 = (end >> 5) + 1;
        r.ns = (sinks + 31) >> 5;
        r.ns = r.ns < r.w0 ? r.ns : r.w0;
    }
    r.nb = r.ns + (end >> 5) - r.w0 + 1;
    return r;
}

// SHARE 4 or 8: the workgroup's waves, as many, share 16 NQ rows and take every SHARE-th block
// of tokens; their results meet in LDS at the end.  SHARE 1: each of four has rows of its own.
// A block and wave are about 335 VALU instructions with two groups (295 with one, 451 with four),
// with 16 rows as with 32, a third of them codes that become operands; so 32 rows where there are
// as many, and three waves a SIMD (two with 32 rows) rather than longer rings: with four stages and
// two waves 16 sequences of up to 8191 take 38 us, 32 so.  Prompts are bound by that issue (69 % of the SIMDs' cycles) and the products (27 %),
// which hardly overlap with two waves; single tokens by no one thing: VALU issue is 49 to 59 % of
// the cycles, products 9 to 14 %, and a wave waits at a wait or barrier for 31 to 43 % of its time
// (the start's dependent loads, a ring of two blocks, the waves' and the parts' uneven ends).
// Measured with heads of 128, 8 of keys and values: these 16, 40 query heads, 32 us with their
// joining (114 MB, 3.6 TB/s); one sequence of 131072, 64 heads, 35 to 36 with it (143 MB, 4.0 TB/s);
// two prompts' 2048 rows, 40 heads, against 6100 tokens 500 to 505 us (528 TFLOP/s).
template <int D, int NG, int NQ, int SHARE>
__global__ __launch_bounds__(SHARE == 8 ? 512 : 256, SHARE == 4 && D < 256 ? 3 : 2) void kv4_attend_kernel(Kv4Cache c, Kv4Batch s, AttendArgs a)
{
    constexpr int NW = D / 32, DT = D / 16, SPG = NW / NG, TPG = DT / NG;
    constexpr bool MERGE = SHARE > 1;
    constexpr int WAVES = MERGE ? SHARE : 4;
    constexpr int ROWS = 16 * NQ, RB = MERGE ? ROWS : 4 * ROWS;
    using RG = Ring<D, NG>;
    static_assert(!MERGE || NQ == 1, "waves that share rows have 16");
    constexpr int LD = D + 4;                              // (a row of the waves' results)
    constexpr int RINGS = WAVES * RG::STAGES * RG::BYTES, SUMS = MERGE ? WAVES * 16 * (LD + 2) * 4 : 0;
    // (one array for all: with several the compiler puts a wait for all loads before each
    // read of the ring)
    __shared__ __attribute__((aligned(16))) uint8_t lds[RINGS > SUMS ? RINGS : SUMS];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, kq = lane >> 4;
    const int H = c.heads, R = a.R;
    uint8_t *const ring = lds + w * (RG::STAGES * RG::BYTES);
    const int cap = s.width << c.shift;                    // tokens that the table has room for
    const int h = blockIdx.x % H, xs = blockIdx.x / H;
    // the rows' block, and the part of the tokens
    const auto row_blocks = [=](const Run &q) { return (q.n * R + RB - 1) / RB; };
    int b, in, of, split = 0, part_blocks = 0;
    Run seq;
    if (MERGE && a.splits > 1) {
        // Parts of one size for all sequences, the longest that a.items of them cover all
        // tokens with: a sequence's last one may be shorter, so as many as there are row blocks are
        // kept back.  (Every wave counts for itself, 64 sequences a step.)
        const auto blocks_of = [=](const Run &q) { return seen_blocks(q.len - q.n, q.len - 1, a.window, a.sinks, cap).nb; };
        long long total = 0;
        int rbs = 0;
        bool huge = false;
        const Run head = kv4_seq(s, lane);                 // (of up to 64 sequences the only load)
        const auto run = [&](int i) { return i < 64 ? head : kv4_seq(s, i); };
        for (int b0 = 0; b0 < s.B; b0 += 64) {
            const Run q = run(b0 + lane);
            const int r = q.n > 0 ? row_blocks(q) : 0, nb1 = r > 0 ? blocks_of(q) : 0;
            huge |= __any((long long)r * nb1 >= 1 << 24);
            total += __builtin_amdgcn_readlane(scan64(huge ? 0 : r * nb1), 63);
            rbs += __builtin_amdgcn_readlane(scan64(r), 63);
        }
        const int spare = a.items - rbs;
        part_blocks = 1 << 28;                             // (too many to count, or no room: no parts)
        if (!huge && total < 1 << 30 && spare > 0)
            part_blocks = (((unsigned)total + spare - 1) / (unsigned)spare + 4) & ~3u;
        const auto parts_of = [=](const Run &q) {
            const int n = (int)((unsigned)(blocks_of(q) + part_blocks - 1) / (unsigned)part_blocks);
            return n < 1 ? 1 : n < a.splits ? n : a.splits;
        };
        if (!find_item(s.B, xs, run, [&](const Run &q) { return row_blocks(q) * parts_of(q); }, b, in, of, seq)) return;
        const int n = parts_of(seq);
        part_blocks = ((blocks_of(seq) + n - 1) / n + 3) & ~3;
        split = in % n;
        in /= n;
        of /= n;
    } else {
        split = xs % a.splits;
        if (!kv4_find(s, xs / a.splits, row_blocks, b, in, of, seq)) return;
    }
    b = __builtin_amdgcn_readfirstlane(b);                 // (the compiler does not see that it is one)
    in = of - 1 - in;                                      // the longest first
    const int rows = seq.n * R;
    const int row0 = in * RB + (MERGE ? 0 : w * ROWS);
    if (row0 >= rows) return;
    const int last = row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1;
    const int first = seq.len - seq.n;                     // position of the first row's token
    const int p0 = first + row0 / R, p1 = first + last / R;

    const SeenBlocks seen = seen_blocks(p0, p1, a.window, a.sinks, cap);
    const int ns = seen.ns, w0 = seen.w0, nb = seen.nb;
    int per = (nb + a.splits - 1) / a.splits;
    if (MERGE) per = a.splits > 1 ? part_blocks : nb;      // (a row block sees no more than its sequence)
    const int j0 = split * per < nb ? split * per : nb, j1 = j0 + per < nb ? j0 + per : nb;

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

    // a wave's blocks: every SHARE-th from j0 + (its number) on
    const int mine = j1 <= j0 ? 0 : (MERGE ? (j1 - j0 - w + SHARE - 1) / SHARE : j1 - j0);
    auto block_of = [&](int i) {
        const int j = j0 + (MERGE ? w : 0) + i * SHARE;
        return j < ns ? j : j - ns + w0;
    };
    // (from the constant address space, for a scalar load: a vector load's wait would be one for
    // the blocks asked for before it, too)
    const __attribute__((address_space(4))) int32_t *const pages =
        (const __attribute__((address_space(4))) int32_t *)(uintptr_t)(s.table + (size_t)b * s.width);
    auto page_of = [&](int i) { return pages[block_of(i) >> (c.shift - 5)]; };
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
        for (int u = 0; u < D / 64; ++u) lds_load16<MERGE ? QG_NT : 0>(c.k + at + u * 256 + lane * 4, to + u * 1024);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) lds_load16<MERGE ? QG_NT : 0>(c.v + at + u * 256 + lane * 4, to + RG::CODES + u * 1024);
        const size_t sat = ((head * NG) << c.shift) + tin;
#pragma unroll
        for (int u = 0; u < SLOADS; ++u) lds_load16<MERGE ? QG_NT : 0>(sz0[u] + sat, to + 2 * RG::CODES + u * 1024);
    };

    // the first block, and the second one's page; whether a block has a page
    bool has = false;
    int next = 0;                                          // the page of the block to be asked for next
    if (mine > 0) {
        const int pg = page_of(0);
        next = page_of(mine > 1 ? 1 : 0);
        has = (unsigned)pg < (unsigned)c.pages;
        load(0, pg);
    }

    // the queries as operands, q' = q 2^(3 - ex) below 8 (64 times their sum is a binary16
    // still); the factor of the scores; the groups' sums as two 16-bit values, against the zeros
    // in the words of lane groups 0 (the upper part) and 1, and -64 times these against the scales
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
        f[n] = bad ? __builtin_nanf("") : ldexpf(a.scale, a.scale_ex + ex - 3);
        float qs[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float sum = 0.0f;
#pragma unroll
            for (int k = g * SPG; k < (g + 1) * SPG; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[k][e] = ldexpf(x[k][e], 3 - ex);
                    sum += x[k][e];
                    qo[n][k][e] = (_Float16)x[k][e];
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            qs[g] = sum;
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
            qz[n][2 * i] = (_Float16)(-OFFSET * (float)part);
            qz[n][2 * i + 1] = part;
        }
    }

    // references; products with the values' codes; with their scales (even rows) and zeros
    // (odd), and with ones (row 2 NG: the sum of p; with eight groups no row is left)
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
    // group g's sum of p vs: row MROW + g, of the same accumulator where there is room
    constexpr int MROW = LROW ? 2 * NG + 1 : 0;
    float4v mid[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) mid[n] = float4v{0, 0, 0, 0};
    int room = ROOM;
    unsigned sixty_four = 0x54005400u;
    asm("" : "+v"(sixty_four));                            // (a register: an instruction takes one constant)

    // all rows see all of a block
    auto sees_all = [&](int t0, bool ok) {
        return ok && t0 + 31 <= p0 && (!a.window || t0 > p1 - a.window || t0 + 31 < a.sinks);
    };
    // (Whether it is so is asked for before the block, where registers are short: the compiler then
    // keeps 214 of them instead of 256 and 18 in memory with four groups of 32 rows, and interleaves less.
    // 2 x 1024 rows of 32 heads against 4096 tokens, groups of 32 of 128 channels: 348 us, 370 the other
    // way; of 256 channels 743 and 824, and 8 x 1 row against 8192 51 and 75.  With fewer groups the other
    // way is faster by up to 6 %.  These 348, 743 and 51 were measured without the look at the scales; with it
    // they are 358, 768 and 51.)
    constexpr bool ASK_FIRST = NG * NQ > 4;
    auto block = [&](bool asked, const uint8_t *x, int t0, bool ok) {
        int ln = lane;                                     // (of many groups: what comes from it is not kept in
        if (NG > 2) asm("" : "+v"(ln));                    // registers)
        const int col = ln & 15, kq = ln >> 4, lane = ln;
        const uint4v *const ksz = reinterpret_cast<const uint4v *>(x + 2 * RG::CODES) + kq;
        const uint4v *const vsz = ksz + NG * 8;
        const unsigned *const kw = reinterpret_cast<const unsigned *>(x + 2 * RG::CODES) + col;
        // the keys' words, and their scales and zeros, all at once
        constexpr bool EARLY = NG * NQ <= 2;               // (more scales and zeros are read when needed)
        constexpr bool EARLY_V = NG * NQ <= 1;
        uint4v kr[2][(NW + 3) / 4], zw[2], sk[2][NG];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t *const kt = x + t * (RG::CODES / 2) + (col * 4 + kq) * (D / 8);
            if constexpr (NW == 2) {
                const uint2v r2 = *reinterpret_cast<const uint2v *>(kt);
                kr[t][0] = uint4v{r2.x, r2.y, 0, 0};
            } else {
#pragma unroll
                for (int i = 0; i < NW / 4; ++i) kr[t][i] = *reinterpret_cast<const uint4v *>(kt + 16 * i);
            }
            zw[t] = uint4v{0, 0, 0, 0};                    // this lane's token: (scale, zero) of four groups
#pragma unroll
            for (int i = 0; i < (NG < 4 ? NG : 4); ++i)
                zw[t][i] = kw[(NG > 4 ? (kq & 1) * 4 + i : i) * 32 + 16 * t];
#pragma unroll
            for (int g = 0; g < (EARLY ? NG : 0); ++g) sk[t][g] = ksz[g * 8 + t * 4];
        }
        __builtin_amdgcn_sched_barrier(0);                 // (not each where it is needed, with a wait of its own)
        float4v sc[NQ][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const auto op = [&](int k) {
                const uint4v r = kr[t][k % (NW / 2) / 2];
                return k % (NW / 2) & 1 ? key_op(r.z, r.w, k >= NW / 2, sixty_four) : key_op(r.x, r.y, k >= NW / 2, sixty_four);
            };
#pragma unroll
            for (int n = 0; n < NQ; ++n)
                sc[n][t] = mfma_f16(__builtin_bit_cast(half8, zw[t]), qz[n], float4v{0, 0, 0, 0});
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                if (!EARLY) {
                    __builtin_amdgcn_sched_barrier(0);
                    sk[t][g] = ksz[g * 8 + t * 4];
                }
                float4v acc[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n) acc[n] = float4v{0, 0, 0, 0};
#pragma unroll
                for (int k = g * SPG; k < (g + 1) * SPG; ++k) {
                    const half8 kc = op(k);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) acc[n] = mfma_f16(kc, qo[n][k], acc[n]);
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sc[n][t][r] = __builtin_fmaf(lo16(sk[t][g][r]), acc[n][r], sc[n][t][r]);
            }
        }
        // the values' words, scales and zeros, on their way while the softmax is taken; za: those of
        // a row of the zeros' product, of which lane (col, kq) takes the halves of one kind of
        // group col / 2, of the eight tokens of lane group kq
        const int zg = col / 2 < NG ? col / 2 : 0;
        const auto values = [&](int u) { return *reinterpret_cast<const uint4v *>(x + RG::CODES + u * 1024 + lane * 16); };
        uint4v vr[D / 64], sv[2][NG], za[2];
#pragma unroll
        for (int u = 0; u < (EARLY ? D / 64 : 0); ++u) vr[u] = values(u);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int g = 0; g < (EARLY_V ? NG : 0); ++g) sv[t][g] = vsz[g * 8 + t * 4];
            za[t] = vsz[zg * 8 + t * 4];
        }
        __builtin_amdgcn_sched_barrier(0);
        // the largest of the values' scales, over all groups and tokens in one lane or another.  (A word's
        // lower half by conversion: a bit cast of a vector's element takes the vector's first one.)
        const auto largest = [&] {
            unsigned short v = (unsigned short)za[0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) v = __builtin_elementwise_max(v, (unsigned short)za[i / 4][i % 4]);
            return v;
        };
        // all rows see all of the block, or some do not: a bit for each score that is hidden.  (A
        // scale that is no number goes that way, too: here it would meet the zeros of the products with
        // ones, and spoil the other groups' sums.)
        bool whole = ASK_FIRST ? asked : sees_all(t0, ok);
        unsigned short large = 0;
        if (!ASK_FIRST && whole) {
            large = largest();
            whole = !__any(large >= 0x7C00);
        }
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
        if (!whole) {
            // a token that one row sees and another does not must not bring it a NaN, nor one group the
            // others: 0 here, and a NaN put in where it is seen; one that no row sees counts for nothing
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = t0 + 16 * t + 4 * kq + r;
                    const bool some = ok && at <= p1 && (!a.window || at > p0 - a.window || at < a.sinks);
                    za[t][r] = !some || odd_word(za[t][r]) ? 0u : za[t][r];
                }
        }
        if (ASK_FIRST || !whole) large = largest();
        bool raise = room > -3 && large > (unsigned)(28 - room) << 10;
        float less = 0.0f;
        if (__any(raise)) {
            int e = large >> 10;                           // vs < 2^(e - 14)
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int other = __shfl_xor(e, o);
                e = other > e ? other : e;
            }
            const int now = 27 - e > -3 ? 27 - e : -3;
            less = (float)(room - now);
            room = now;
        }
        float mx[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            float v = fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3]));
            v = fmaxf(v, fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3])));
            mx[n] = v * f[n];                              // (f > 0)
            raise |= mx[n] > m[n] + (SLACK + (float)room);
        }
        if (__any(raise)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float v = fmaxf(mx[n], __shfl_xor(mx[n], 16));
                v = fmaxf(m[n] + less, fmaxf(v, __shfl_xor(v, 32)) - (float)room);
                const float by = __builtin_amdgcn_exp2f(m[n] - v);
                m[n] = v;
                l[n] *= by;
                z[n] *= by;
                if (!LROW) mid[n] *= by;
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

        uint4v zh;
        const unsigned sel = (col & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            zh[2 * t] = __builtin_amdgcn_perm(za[t][1], za[t][0], sel);
            zh[2 * t + 1] = __builtin_amdgcn_perm(za[t][3], za[t][2], sel);
        }
        if (LROW && col >= 2 * NG) {                       // (rows behind that of the ones: nothing)
            const unsigned w1 = col == 2 * NG ? 0x3C003C00u : 0u;
            zh = uint4v{w1, w1, w1, w1};
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) z[n] = mfma_f16(__builtin_bit_cast(half8, zh), pf[n], z[n]);

#pragma unroll
        for (int g = 0; g < NG; ++g) {
            uint4v sz[2];
            if (!EARLY_V) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 2; ++t) sz[t] = EARLY_V ? sv[t][g] : vsz[g * 8 + t * 4];
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
            if (!EARLY)
#pragma unroll
                for (int u = (g * TPG + 3) / 4; u < ((g + 1) * TPG + 3) / 4; ++u) vr[u] = values(u);
            half8 po[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) po[n][4 * t + r] = (_Float16)__builtin_fmaf(lo16(sz[t][r]), sc[n][t][r], 0.0f);
            const unsigned one = col == MROW + g ? 0x3C003C00u : 0u;
            const half8 ones = __builtin_bit_cast(half8, uint4v{one, one, one, one});
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float4v &to = LROW ? z[n] : mid[n];
                to = mfma_f16(ones, po[n], to);
            }
#pragma unroll
            for (int d = g * TPG; d < (g + 1) * TPG; ++d) {
                const half8 vo = value_op(vr[d / 4][d % 4], sixty_four);
#pragma unroll
                for (int n = 0; n < NQ; ++n) o[n][d] = mfma_f16(vo, po[n], o[n][d]);
            }
        }
    };

    for (int i = 0; i < mine; ++i) {
        const int more = mine - 1 - i;                     // blocks behind this one
        const bool ok = has;
        if (more > 0) {
            has = (unsigned)next < (unsigned)c.pages;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage's last reads are done
            load(i + 1, next);
            debug_stage_sync();
            wait_loads<RG::LOADS>();
            __builtin_amdgcn_sched_barrier(0);             // (behind that wait, or it waits for this load)
            next = page_of(more > 1 ? i + 2 : i);
        } else {
            wait_loads<0>();
        }
        const int t0 = block_of(i) << 5;
        const uint8_t *const x = ring + (i % RG::STAGES) * RG::BYTES;
        bool asked = false;
        if (ASK_FIRST) {
            const unsigned *const scales = reinterpret_cast<const unsigned *>(x + 2 * RG::CODES) + 32 * NG;
            bool odd = false;
#pragma unroll
            for (int u = 0; u < NG / 2; ++u) odd |= (scales[64 * u + lane] & 0x7C00u) == 0x7C00u;
            asked = sees_all(t0, ok) && !__any(odd);
        }
        block(asked, x, t0, ok);
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
            const float zs = __shfl(zz[g % 2], 16 * (g / 2) + col) -
                             (OFFSET + 8.0f) * __shfl((LROW ? z : mid)[n][(MROW + g) % 4], 16 * ((MROW + g) / 4) + col);
#pragma unroll
            for (int d = g * TPG; d < (g + 1) * TPG; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[n][d][r] += zs;
        }
    }

    const size_t all = (size_t)s.T * a.q_heads;
    if constexpr (MERGE) {
        float(*const so)[16][LD] = reinterpret_cast<float(*)[16][LD]>(lds);
        float(*const sm)[16] = reinterpret_cast<float(*)[16]>(lds + WAVES * 16 * LD * 4), (*const sl)[16] = sm + WAVES;
        __syncthreads();                                   // (the waves' rings are done with)
        // what a thread adds up: four channels of a row
        constexpr int TPR = D / 4, PASS = 64 * WAVES / TPR;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<float4v *>(&so[w][col][16 * d + 4 * kq]) = o[0][d];
        if (kq == 0) {
            sm[w][col] = m[0];
            sl[w][col] = l[0];
        }
        debug_stage_sync();
        __syncthreads();
        for (int r = threadIdx.x / TPR; r < 16 && row0 + r < rows; r += PASS) {
            const int ch = threadIdx.x % TPR * 4;
            float mm = sm[0][r];
#pragma unroll
            for (int i = 1; i < WAVES; ++i) mm = fmaxf(mm, sm[i][r]);
            float sum = 0.0f;
            float4v acc = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                const float by = __builtin_amdgcn_exp2f(sm[i][r] - mm);
                sum += by * sl[i][r];
                acc += by * *reinterpret_cast<const float4v *>(&so[i][r][ch]);
            }
            const int rr = row0 + r, i = rr / R;
            const size_t g = ((size_t)seq.row + i) * a.q_heads + (size_t)h * R + (rr - i * R);
            if (a.splits > 1) {
                if (ch == 0 && split == 0) a.parts[g] = per < nb ? (nb + per - 1) / per : 1;
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
    } else {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            if (row0 + 16 * n + col >= rows) continue;
            if (a.splits > 1) {
                if (kq == 0) {
                    if (split == 0) a.parts[grow[n]] = a.splits;
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
// without a token hold sum 0 and no values.  Bound by latency: the number of parts, their maxima,
// then all values at once (640 rows 4.6 us).
constexpr int MAX_SPLITS = 128;
template <int D>
__global__ __launch_bounds__(512) void kv4_join_kernel(Kv4Batch s, AttendArgs a)
{
    constexpr int TPR = D / 4, GR = 512 / TPR, MOST = (MAX_SPLITS + GR - 1) / GR;
    const size_t all = (size_t)s.T * a.q_heads, g = blockIdx.x;
    if (s.off) {                                          // rows of no sequence stay as they are
        const long long t = (long long)(g / a.q_heads);
        if (t < s.off[0] || t >= s.off[s.B]) return;
    }
    const int tid = threadIdx.x, grp = tid / TPR, ch = tid % TPR * 4;
    __shared__ float4v so[GR][TPR];
    __shared__ float by[MAX_SPLITS], top[2], total[2];
    int n = a.parts[g];
    n = n < 0 ? 0 : n < a.splits ? n : a.splits;
    // (two waves hold the parts)
    float mi = NONE, li = 0.0f;
    if (tid < n) {
        mi = a.ml[(tid * all + g) * 2];
        li = a.ml[(tid * all + g) * 2 + 1];
    }
    float4v v[MOST];
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int k = grp + i * GR;                        // (past the last: read again, weight 0)
        v[i] = *reinterpret_cast<const float4v *>(a.part + ((k < n ? k : 0) * all + g) * D + ch);
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
        // a part without a token has no values to be read: -1.  (Others are added also where their weight
        // is 0: they may be no numbers.)
        by[tid] = li == 0.0f ? -1.0f : e;
        li = li == 0.0f ? 0.0f : li * e;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) li += __shfl_xor(li, o);
        if (tid % 64 == 0) total[tid / 64] = li;
    }
    debug_stage_sync();
    __syncthreads();
    float4v acc = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int k = grp + i * GR;
        const float e = k < MAX_SPLITS ? by[k] : -1.0f;
        if (!(e < 0.0f)) acc += e * v[i];
    }
    so[grp][tid % TPR] = acc;
    debug_stage_sync();
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 1; i < GR; ++i) acc += so[i][tid];
    const float sum = total[0] + total[1];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = a.bf16 ? f2bf(acc[e] * inv) : f2h(acc[e] * inv);
    *reinterpret_cast<uint2v *>(a.out + g * D + ch) = uint2v{r[0] | (uint32_t)r[1] << 16, r[2] | (uint32_t)r[3] << 16};
}

template <int D, int NG>
void launch_attend(const Kv4AttendPlan &p, const Kv4Cache &c, const Kv4Batch &s, const AttendArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)p.workgroups);
    if (p.shared == 8) {
        if constexpr (D < 256)
            hipLaunchKernelGGL((kv4_attend_kernel<D, NG, 1, 8>), grid, dim3(512), 0, st, c, s, a);
    } else if (p.shared)
        hipLaunchKernelGGL((kv4_attend_kernel<D, NG, 1, 4>), grid, dim3(256), 0, st, c, s, a);
    else
        hipLaunchKernelGGL((kv4_attend_kernel<D, NG, D == 256 ? 1 : 2, 1>), grid, dim3(256), 0, st, c, s, a);
}

} // namespace

// Decode batches (up to 16 rows of a key/value head in a sequence): the four or eight waves
// of a workgroup share the rows.  More rows: each wave has 32 of its own (16 of 256 channels).
Kv4AttendPlan kv4_attend_plan(int T, int max_new, int B, int q_heads, int heads, int D, int max_tokens, int window,
                              int sinks)
{
    Kv4AttendPlan p;
    const long long R = q_heads / heads;
    p.shared = max_new * R <= 16 ? 4 : 0;
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
    // Parts along the tokens where the rows alone do not fill the CUs once (with three workgroups
    // each of shared rows up to 128 channels, else two), of at least a block of tokens for each
    // wave.  Rows that a workgroup's waves share are cut into parts of one size (the kernel
    // finds it), the others each into as many.
    const long long most = (tokens + 127) / 128, fit = p.shared && D < 256 ? 768 : 512;
    // (More rows than the joining launch has threads for would be enough work whole, and are here only
    // with a max_new far below the truth.)
    const bool may_join = (long long)T * q_heads < 1 << 22;
    p.splits = 1;
    p.items = 0;
    if (p.shared) {
        long long n = fit / heads;
        n = n < some * most ? n : some * most;
        // (joining them costs 5 us: not for fewer than two parts each of few tokens; 64 sequences
        // that see 1000 tokens each take 36 us in 96 parts, 26.5 whole.  Of many tokens a
        // sequence may be far longer than the others: the table's width is all that is known here, and
        // these 64 take 31 us instead of 21 where it has room for more than 4096.)
        // Few tokens: eight waves against four in parts and a second kernel, where the workgroups have a
        // CU each.  1, 4, 16 and 32 sequences of 8 heads of 128, us in a graph, eight waves and parts: 768
        // tokens 9.7/10.8, 9.8/11.0, 9.9/13.7, 10.3/16.6; 1024 11.1/10.8, 11.2/11.1, 11.4/13.8,
        // 11.8/18.1; 1280 12.4/10.8, 12.7/11.1, 12.9/15.4, 13.3/19.7; 1536 14.0/10.8, 14.3/11.1,
        // 14.6/15.6, 14.8/21.2.  Called one by one the second kernel and its workspace cost the host
        // more: 14.7 at every length, and eight waves are faster up to 1536.  The border lies between the
        // two ways of calling.
        const bool eight = D < 256 && likely <= 256 && tokens <= 1280;
        if (eight) p.shared = 8;
        if (!eight && may_join && (n >= 2 * some || (n > some && tokens > 4096))) {
            p.items = (int)n;
            n = n - some + 1;
            p.splits = (int)(n < MAX_SPLITS ? n : MAX_SPLITS);
            // (no part may be numbered past them: fewer items, longer parts)
            if (p.items > p.splits + some - 1) p.items = (int)(p.splits + some - 1);
        }
        if (p.splits == 1) p.items = 0;
    } else {
        long long n = fit / likely;
        n = n > most ? most : n;
        n = n > MAX_SPLITS ? MAX_SPLITS : n;
        p.splits = n < 1 || !may_join ? 1 : (int)n;
    }
    p.workgroups = (p.items ? (p.items > blocks ? p.items : blocks) : blocks * p.splits) * heads;
    p.bytes = p.splits == 1 ? 0 : (size_t)T * q_heads * ((size_t)p.splits * (D + 2) + 1) * sizeof(float);
    return p;
}

hipError_t launch_kv4_attend(const Kv4AttendPlan &p, const Kv4Cache &c, const Kv4Batch &s, const void *q, long long ldq,
                             int q_heads, int dtype, float scale, int window, int sinks, void *out, void *ws,
                             hipStream_t st)
{
    const size_t all = (size_t)s.T * q_heads;
    float *const part = (float *)ws;
    int scale_ex;
    const float log2_scale = frexpf(scale, &scale_ex) * 1.4426950408889634f;
    const AttendArgs a = {(const uint16_t *)q, (uint16_t *)out, ldq, q_heads, q_heads / c.heads, dtype == QG_DT_BF16,
                          log2_scale, scale_ex, window, sinks, p.splits, p.items, part,
                          part ? part + (size_t)p.splits * all * c.D : nullptr,
                          part ? (int32_t *)(part + (size_t)p.splits * all * (c.D + 2)) : nullptr};
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
    case 64: hipLaunchKernelGGL((kv4_join_kernel<64>), dim3((unsigned)all), dim3(512), 0, st, s, a); break;
    case 128: hipLaunchKernelGGL((kv4_join_kernel<128>), dim3((unsigned)all), dim3(512), 0, st, s, a); break;
    default: hipLaunchKernelGGL((kv4_join_kernel<256>), dim3((unsigned)all), dim3(512), 0, st, s, a); break;
    }
    return hipGetLastError();
}

} // namespace qg
