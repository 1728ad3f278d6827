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
#include <cstring>

#include "qg_device.h"
#include "qg_launch.h"

namespace qg {
namespace {

constexpr int KB8 = 128;   // k extent of a scale block, bytes of a tile row

// An offset past every buffer range here (a block's rows, or with a row index all
// of A: at most 2^32 - 2^23 bytes, which the caller checks) that does not wrap when
// a step's scalar offset is added.  Those go past the last of the at most 2^15 k blocks by
// the steps asked for ahead: MAX_AHEAD bounds them, and each kernel checks its own.
constexpr unsigned FP8_PAST = 0xFFBFFFF0u - 0x1000u;
constexpr int MAX_AHEAD = 16;
static_assert(FP8_PAST > 0xFFFFFFFFu - (1u << 23) && (1u << 15) * KB8 + MAX_AHEAD * KB8 + 16 <= 0xFFFFFFFFu - FP8_PAST,
              "past every range, and no wrap");
// The same for a tile of W: at most 256 rows, 2^30 bytes, and scalar offsets
// up to such a tile.
constexpr unsigned FP8_W_PAST = 0x80000000u;

// The BM-row blocks of all experts, in order, and the one an index names.  The
// counts stand in the device's offsets, so the grid is an upper bound and every
// wave scans them for itself, 64 experts a step.
struct RowBlock {
    int e, m0, m1;      // expert, first row, end of the expert's rows
};

__device__ inline void expert_rows(const int32_t *__restrict__ offsets, int E, int M, int e, int &r0,
                                   int &r1)
{
    r0 = r1 = 0;
    if (e < E) {
        r0 = offsets[e];
        r1 = offsets[e + 1];
        r0 = r0 < 0 ? 0 : (r0 > M ? M : r0);
        r1 = r1 < r0 ? r0 : (r1 > M ? M : r1);
    }
}

// Inclusive scan of the row blocks of 64 experts from e0 on, one a lane.
struct RowScan {
    int r0, r1, blocks, sum;
};

__device__ inline RowScan scan_rows(const int32_t *__restrict__ offsets, int E, int M, int BM, int e0)
{
    const int lane = threadIdx.x & 63;
    RowScan s;
    expert_rows(offsets, E, M, e0 + lane, s.r0, s.r1);
    s.blocks = (s.r1 - s.r0 + BM - 1) / BM;
    s.sum = s.blocks;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(s.sum, o);
        if (lane >= o) s.sum += v;
    }
    return s;
}

__device__ inline int row_block_count(const int32_t *__restrict__ offsets, int E, int M, int BM,
                                      const RowScan &first)
{
    if (!offsets) return (M + BM - 1) / BM;
    int n = __builtin_amdgcn_readlane(first.sum, 63);
    for (int e0 = 64; e0 < E; e0 += 64)
        n += __builtin_amdgcn_readlane(scan_rows(offsets, E, M, BM, e0).sum, 63);
    return n;
}

// Row block rb, or the expert it belongs to (m0 its first row, `before` the
// row blocks of the experts before it, `blocks` its own); no rows if there are fewer.
// first: scan_rows from expert 0 on.
struct ExpertRows {
    int e, m0, m1, before, blocks;
};
__device__ inline ExpertRows find_expert(const int32_t *__restrict__ offsets, int E, int M, int BM,
                                         int rb, const RowScan &first)
{
    if (!offsets) return ExpertRows{0, 0, M, 0, (M + BM - 1) / BM};
    RowScan s = first;
    int base = 0;
    for (int e0 = 0;;) {
        const unsigned long long hit = __ballot(base + s.sum > rb);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            return ExpertRows{e0 + l, __builtin_amdgcn_readlane(s.r0, l), __builtin_amdgcn_readlane(s.r1, l),
                              base + __builtin_amdgcn_readlane(s.sum - s.blocks, l),
                              __builtin_amdgcn_readlane(s.blocks, l)};
        }
        base += __builtin_amdgcn_readlane(s.sum, 63);
        e0 += 64;
        if (e0 >= E) return ExpertRows{0, 0, 0, 0, 0};
        s = scan_rows(offsets, E, M, BM, e0);
    }
}
__device__ inline RowBlock find_rows(const int32_t *__restrict__ offsets, int E, int M, int BM,
                                     int rb, const RowScan &first)
{
    const ExpertRows x = find_expert(offsets, E, M, BM, rb, first);
    if ((unsigned)(rb - x.before) >= (unsigned)x.blocks) return RowBlock{0, 0, 0};
    return RowBlock{x.e, x.m0 + (rb - x.before) * BM, x.m1};
}

// The tile of workgroup b out of rbs row blocks x nbn column blocks, false if
// there is none.  Workgroups go to the eight XCDs in turn; each XCD takes a
// contiguous run of the tiles, ordered expert by expert and in bands of 1536 of an
// expert's rows, so that the tiles an XCD computes at a time share both operands in
// its L2.  4096 tokens to 8 of 64 experts at 2048 x 7168: 610 us (bands of 1024
// rows 621; bands that run over the experts' borders 647), dense no difference.
template <int BM>
__device__ inline bool tile_of(int b, const int32_t *__restrict__ offsets, int E, int M, int nbn,
                               RowBlock &blk, int &nb)
{
    constexpr int GM = 1536 / BM;
    RowScan scan = {};
    if (offsets) scan = scan_rows(offsets, E, M, BM, 0);
    const int tiles = row_block_count(offsets, E, M, BM, scan) * nbn;
    if (b >= tiles) return false;
    const int x = b & 7, q = tiles >> 3, r = tiles & 7;
    const int id = x * q + (x < r ? x : r) + (b >> 3);
    const ExpertRows rows = find_expert(offsets, E, M, BM, id / nbn, scan);
    const int of = id - rows.before * nbn;
    if ((unsigned)of >= (unsigned)(rows.blocks * nbn)) return false;      // (offsets that are none)
    const int band = of / (GM * nbn), in = of - band * (GM * nbn);
    const int high = rows.blocks - band * GM < GM ? rows.blocks - band * GM : GM;
    nb = in / high;
    blk = RowBlock{rows.e, rows.m0 + (band * GM + in - nb * high) * BM, rows.m1};
    return true;
}

template <bool BF16>
__device__ inline uint16_t out16(float f) { return BF16 ? f2bf(f) : f2h(f); }

// Four consecutive columns n .. n + 3 of a row; zeros for a row of no activations.
template <bool BF16>
__device__ inline void store4(uint16_t *c, float4v x, bool zero, int n, int N, bool wide)
{
    uint16_t h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = zero ? 0 : out16<BF16>(x[r]);
    if (wide) {
        if (n < N) *reinterpret_cast<uint2v *>(c) = uint2v{h[0] | (unsigned)h[1] << 16, h[2] | (unsigned)h[3] << 16};
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < N) c[r] = h[r];
    }
}

// ---- tiled kernel ----
// BM x BN tile per workgroup of WM x WN waves; each wave MT x NT 16 x 16
// tiles.  A 128-k step of both operands (rows of 128 bytes) is loaded straight
// to LDS, double-buffered, one barrier a step.  In LDS, 16-byte chunk c of row r
// stands at position c ^ (r % 8), so that the 16 rows a wave reads at once
// spread over the banks.
// KS > 1: KS such groups of waves, each with LDS of its own, take the steps in
// turn, and their sums meet in LDS in the order of the groups; for grids that
// leave CUs idle or K long, where a step's latency is what counts.
// 4096 x 5120 x 17408 (M x K x N): 332 to 348 us, 2.1 to 2.2 PFLOP/s of the 3.45 that
// MFMAs with four FMAs each reach from registers alone; a third of the waves' time is
// spent at the step's barrier, for loads that come from beyond L2 (with L2 hits only 10 %
// faster).
// b: the workgroup's number among those of this tile.
template <int BM, int BN, int WM, int WN, int KS, bool BF16>
__device__ __forceinline__ void fp8_tile(
    const uint8_t *__restrict__ Aall, const float *__restrict__ a_scale,
    const int32_t *__restrict__ a_rows, int M_a, const uint8_t *__restrict__ Wall,
    const float *__restrict__ Sall, const int32_t *__restrict__ offsets, int E, int M, int N,
    int K, int KB, int NB, int col_first, int nbn, uint16_t *__restrict__ C, int b)
{
    constexpr int NW = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
    constexpr int LA = BM / 8 / NW, LW = BN / 8 / NW;    // 1 KB loads per wave and step
    static_assert(LA * NW * 8 == BM && LW * NW * 8 == BN, "whole loads per wave");
    // (KS groups' steps end within KS - 1 blocks past the last, two more steps are asked for)
    static_assert(3 * KS - 1 <= MAX_AHEAD, "the scalar offset of the last load");
    static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0, "a wave's columns share one weight scale");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds_all[];
    constexpr int STAGE = (BM + BN) * KB8;

    int n0;
    RowBlock blk;
    // uniform over the workgroup, before any barrier
    if (!tile_of<BM>(b, offsets, E, M, nbn, blk, n0)) return;
    n0 = col_first + n0 * BN;
    const int e = __builtin_amdgcn_readfirstlane(blk.e);
    const int m0 = __builtin_amdgcn_readfirstlane(blk.m0);
    const int m1 = __builtin_amdgcn_readfirstlane(blk.m1);
    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = KS > 1 ? wave_all / NW : 0, wave = KS > 1 ? wave_all % NW : wave_all;
    const int wm = wave / WN, wn = wave % WN;
    uint8_t *lds = lds_all + group * (2 * STAGE);
    // this group's steps: kt stands for k block kt * KS + group
    const int steps = (KB + KS - 1) / KS;

    // every lane's source chunk within a row, and its rows' byte offsets; rows
    // past the end read the last row (never stored)
    const int chunk = (lane & 7) ^ (lane >> 3);
    const int rows_n = N - n0 < BN ? N - n0 : BN, rows_m = m1 - m0 < BM ? m1 - m0 : BM;
    const uint8_t *W = Wall + ((size_t)e * N + n0) * K;
    const __amdgpu_buffer_rsrc_t w_rs = buffer_rsrc(W, (size_t)rows_n * K);
    const __amdgpu_buffer_rsrc_t a_rs =
        a_rows ? buffer_rsrc(Aall, (size_t)M_a * K) : buffer_rsrc(Aall + (size_t)m0 * K, (size_t)rows_m * K);
    unsigned a_off[LA];
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
    // (rows of W past N read nothing: zeros, never stored)
    const unsigned w_off = (unsigned)(wave * LW * 8 + (lane >> 3)) * (unsigned)K + chunk * 16;
    // Every load of step kt.  Chunks past the end of K (in the last step of a
    // K that is no multiple of 128, and in the steps past the last that the loop
    // below asks for without a branch) take an offset beyond every range, which
    // the step's scalar offset cannot wrap: such loads give zeros and read
    // nothing.
    // (plain variables of a fixed type: a target builtin given an argument
    // whose type depends on a template parameter loses the kernel's host
    // launch stub)
    constexpr int PIECES = LA + LW;
    auto load_piece = [&](int kt, int q) {
        const int k = (kt * KS + group) * KB8;
        const bool in = k + chunk * 16 < K;
        // (pinned: one load for all lanes, not two under half an exec mask)
        if (q < LA) {
            unsigned off = in ? a_off[q] : FP8_PAST;
            pin(off);
            uint8_t *dst = lds + (kt & 1) * STAGE + (wave * LA + q) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rs, (__attribute__((address_space(3))) void *)dst, 16, off, k, 0, 0);
        } else {
            unsigned off = in ? w_off : FP8_W_PAST;
            pin(off);
            uint8_t *dst = lds + (kt & 1) * STAGE + (BM / 8 + wave * LW + q - LA) * 1024;
            const int more = k + (q - LA) * 8 * K;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rs, (__attribute__((address_space(3))) void *)dst, 16, off, more, 0, 0);
        }
        // (the waiting build: each load lands before the next MFMA, none at the barrier)
        debug_stage_sync();
    };

    // Scales, four steps at a time: lane l loads, for its row (l % 16) of each
    // m-tile, the scale of step 4 c + l / 16, so one 4-byte load a row serves
    // four steps (a load for every step asks L2 for a whole line per row each
    // time: 52 of 278 us at 4096 x 8192 x 8192).  The product with the
    // weight block's scale is then handed to the four lanes of a row through
    // LDS.
    // The rows' scale offsets stand in LDS, where they cost no registers of the main
    // loop; bit 0 marks a row of no activations.
    unsigned *s_tab = reinterpret_cast<unsigned *>(lds_all + KS * 2 * STAGE);
    for (int i = threadIdx.x; i < BM; i += 64 * NW * KS) {
        int r = m0 + i < m1 ? i : m1 - 1 - m0;
        bool none = false;
        if (a_rows) {
            r = a_rows[m0 + r];
            none = (unsigned)r >= (unsigned)M_a;
            r = none ? 0 : r;
        }
        s_tab[i] = (unsigned)r * (unsigned)KB * 4u | (none ? 1u : 0u);
    }
    __syncthreads();
    const int my_row = wm * MT * 16 + (lane & 15);     // of m-tile 0
    const __amdgpu_buffer_rsrc_t sa_rs = a_rows ? buffer_rsrc(a_scale, (size_t)M_a * KB * 4)
                                                : buffer_rsrc(a_scale + (size_t)m0 * KB, (size_t)rows_m * KB * 4);
    int nb = (n0 + wn * NT * 16) / 128;
    nb = nb < NB ? nb : NB - 1;
    const __amdgpu_buffer_rsrc_t sw_rs = buffer_rsrc(Sall + ((size_t)e * NB + nb) * KB, (size_t)KB * 4);

    float4v acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};

    // operand position of this lane in a 16-row tile: chunks q and q ^ 4 of
    // lane group q = lane / 16
    const int o0 = (lane & 15) * KB8 + (((lane >> 4) ^ (lane & 7)) * 16);
    const int a_base = wm * MT * 16 * KB8, w_base = (BM + wn * NT * 16) * KB8;
    auto operand = [&](int pos) {      // byte position of a 16-row tile in LDS
        const int4v lo = *reinterpret_cast<const int4v *>(lds + pos + o0);
        const int4v hi = *reinterpret_cast<const int4v *>(lds + pos + (o0 ^ 64));
        return int8v{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    };

    // Schedule.  One wave's MFMAs follow each other without a pause only if
    // nothing it issues in between waits: the FMAs that fold a product run two
    // MFMAs behind it (ring of four products), the next column tile's operand is
    // read a column tile ahead, and the step's one barrier stands before its last
    // column tile.  There every operand of the step is in registers, so behind it
    // the step's buffer is filled again (for step k + 2), step k + 1's tiles have
    // landed, and its first operands are read between the last MFMAs.  The
    // scheduling barriers and the pinned values keep this order (without the pins the
    // compiler delays FMAs, keeps their products alive and spills).
    float sa[MT], sb;             // scales of the next four steps, in flight
    float s[MT], s_old[MT];       // this step's, and those of the step whose last results wait
    float4v p[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) p[t] = float4v{0.f, 0.f, 0.f, 0.f};
    auto load_scales = [&](int c) {
        // (with KS > 1 a block past the last may be multiplied: its scale is 0; with
        // one group it never is)
        const bool in = KS == 1 || (c * 4 + (lane >> 4)) * KS + group < KB;
        const unsigned o = in ? (unsigned)((lane >> 4) * KS + group) * 4u : FP8_PAST;
        sb = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(sw_rs, o, c * 16 * KS, 0));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const unsigned os = in ? (s_tab[my_row + 16 * t] & ~1u) + ((lane >> 4) * KS + group) * 4 : FP8_PAST;
            sa[t] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(sa_rs, os, c * 16 * KS, 0));
        }
    };
    // the products of the scales of four steps, [m-tile][step][row] of this wave's own
    float *four = reinterpret_cast<float *>(lds_all + KS * 2 * STAGE + BM * 4) + wave_all * (MT * 64);
    auto keep_scales = [&]() {
#pragma unroll
        for (int t = 0; t < MT; ++t) four[t * 64 + lane] = sa[t] * sb;
    };
    auto of_step = [&](int t, int at) { return four[t * 64 + (at & 3) * 16 + (lane & 15)]; };
    if (m0 + wm * MT * 16 >= m1) {
        // None of this wave's rows exist (the last block of an expert's rows): it
        // keeps loading and meeting the others at the barriers, and leaves the
        // matrix cores to them.
#pragma unroll
        for (int q = 0; q < PIECES; ++q) load_piece(0, q);
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
#pragma unroll
        for (int q = 0; q < PIECES; ++q) load_piece(1, q);
        for (int kt = 0; kt < steps; ++kt) {
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
            __syncthreads();
#pragma unroll
            for (int q = 0; q < PIECES; ++q) load_piece(kt + 2, q);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
        if (KS > 1) {
            __syncthreads();
            __syncthreads();
        }
        return;
    }
    load_scales(0);
#pragma unroll
    for (int q = 0; q < PIECES; ++q) load_piece(0, q);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) s_old[t] = 0.f;
    keep_scales();
#pragma unroll
    for (int t = 0; t < MT; ++t) s[t] = of_step(t, 0);
    // Loads go out one behind each of the first MFMAs after the barrier: in one
    // burst behind it they hold every wave's issue until the address unit has
    // taken them (289 against 278 us at 4096 x 8192 x 8192), and further apart
    // they land late (243 against 237).  Slot i is behind MFMA i of the last column
    // tile, slot (j + 1) * MT + i behind MFMA i of column tile j of the next step.
    static_assert(PIECES <= NT * MT, "every load has a slot");
#pragma unroll
    for (int i = 0; i < MT; ++i)
        if (i < PIECES) load_piece(1, i);
    int8v a[MT], w[2];
    w[0] = operand(w_base);
#pragma unroll
    for (int i = 0; i < MT; ++i) a[i] = operand(a_base + i * 16 * KB8);
    static_assert(NT % 2 == 0 && MT * NT % 4 == 0, "rings of two operands and four products");

    // one step; at = kt % 4, a constant at each call
    auto step = [&](int kt, int at) __attribute__((always_inline)) {
        const int cur = (at & 1) * STAGE, nxt = STAGE - cur;
        float s_new[MT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (j == NT - 1) {
                // every load of step kt + 1 has landed and every read of step kt is done
                __builtin_amdgcn_s_waitcnt(0);
                __syncthreads();
                if (at == 3) keep_scales();
#pragma unroll
                for (int t = 0; t < MT; ++t) s_new[t] = of_step(t, at + 1);
                if (at == 2) load_scales((kt >> 2) + 1);
                w[0] = operand(nxt + w_base);      // (stale data after the last step, unused)
            } else {
                w[(j + 1) & 1] = operand(cur + w_base + (j + 1) * 16 * KB8);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int t = j * MT + i, u = t - 2;      // this tile, the tile folded now
                p[t & 3] = mfma_fp8(w[j & 1], a[i], float4v{0.f, 0.f, 0.f, 0.f});
                pin(p[t & 3]);
                const int ui = u < 0 ? (u + MT * NT) % MT : u % MT, uj = u < 0 ? (u + MT * NT) / MT : u / MT;
                const float us = u < 0 ? s_old[ui] : s[ui];
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[ui][uj][r] = __builtin_fmaf(p[u & 3][r], us, acc[ui][uj][r]);
                pin(acc[ui][uj]);
                const int slot = j == NT - 1 ? i : (j + 1) * MT + i;
                if (slot < PIECES) load_piece(j == NT - 1 ? kt + 2 : kt + 1, slot);
                if (j == NT - 1) a[i] = operand(nxt + a_base + i * 16 * KB8);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            s_old[t] = s[t];
            s[t] = s_new[t];
        }
    };
    // Four steps to a round, for the scales, then the up to three left over.  (No
    // branch inside a step, where the compiler would sink the FMAs before it to
    // where it joins again and keep all products alive, and no way out of the
    // middle of a round, which costs copies of the accumulators.)
    int kt = 0;
    for (; kt + 4 <= steps; kt += 4) {
        step(kt, 0);
        step(kt + 1, 1);
        step(kt + 2, 2);
        step(kt + 3, 3);
    }
    if (kt < steps) {
        step(kt, 0);
        if (kt + 1 < steps) {
            step(kt + 1, 1);
            if (kt + 2 < steps) step(kt + 2, 2);
        }
    }
#pragma unroll
    for (int u = MT * NT - 2; u < MT * NT; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            acc[u % MT][u / MT][r] = __builtin_fmaf(p[u & 3][r], s_old[u % MT], acc[u % MT][u / MT][r]);

    // The tile goes out through LDS: a lane holds four columns of one row, so that
    // storing from registers would write 32 bytes of a 128-byte line at a time.  Each
    // wave lays its own rows out (chunk c of 16 bytes of row r at c ^ (r % 16),
    // against bank conflicts) and writes them 16 bytes a lane.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));     // the last (empty) loads to LDS, of every wave
    __syncthreads();
    constexpr int ROW = NT * 16 * 2, CH = ROW / 16, RPI = 64 / CH;   // bytes and chunks of a row, rows of one store
    static_assert(MT * 16 * ROW * NW <= 2 * STAGE && CH >= 2 && CH <= 16, "the tile fits, a row in 16 chunks");
    if (KS > 1) {
        constexpr int PART = MT * NT * NW * 64;       // float4 of one group
        static_assert((KS - 1) * PART * 16 <= KS * 2 * STAGE, "the groups' sums fit");
        float4v *part = reinterpret_cast<float4v *>(lds_all);
        if (group > 0) {
#pragma unroll
            for (int t = 0; t < MT * NT; ++t)
                part[(group - 1) * PART + (t * NW + wave) * 64 + lane] = acc[t / NT][t % NT];
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int g = 1; g < KS; ++g)
#pragma unroll
                for (int t = 0; t < MT * NT; ++t) acc[t / NT][t % NT] += part[(g - 1) * PART + (t * NW + wave) * 64 + lane];
        }
        __syncthreads();
        if (group > 0) return;
    }
    const int row0 = m0 + wm * MT * 16, col0 = n0 + wn * NT * 16;
    bool bad[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) bad[i] = s_tab[my_row + 16 * i] & 1u;
    if (N % 8 == 0 && ((uintptr_t)C & 15) == 0) {
        uint8_t *mine = lds + wave * (MT * 16 * ROW);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint16_t h[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) h[r] = bad[i] ? 0 : out16<BF16>(acc[i][j][r]);
                const int r = i * 16 + (lane & 15), c = j * 2 + (lane >> 5);
                *reinterpret_cast<uint2v *>(mine + r * ROW + ((c ^ r) & (CH - 1)) * 16 + ((lane >> 4) & 1) * 8) =
                    uint2v{h[0] | (unsigned)h[1] << 16, h[2] | (unsigned)h[3] << 16};
            }
        // (the wave reads back its own words, in order)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        debug_stage_sync();
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int k = 0; k < MT * 16 / RPI; ++k) {
            const int r = k * RPI + lane / CH, c = lane % CH;
            const uint4v v = *reinterpret_cast<const uint4v *>(mine + r * ROW + ((c ^ r) & (CH - 1)) * 16);
            if (row0 + r < m1 && col0 + c * 8 < N)
                __builtin_nontemporal_store(v, reinterpret_cast<uint4v *>(C + (size_t)(row0 + r) * N + col0 + c * 8));
        }
        return;
    }
    const bool wide = N % 4 == 0 && ((uintptr_t)C & 7) == 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = row0 + i * 16 + (lane & 15);
        if (m >= m1) continue;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = col0 + j * 16 + 4 * (lane >> 4);
            store4<BF16>(C + (size_t)m * N + n, acc[i][j], bad[i], n, N, wide);
        }
    }
}

template <int BM, int BN, int WM, int WN, int KS, bool BF16>
__global__ __launch_bounds__(64 * WM * WN * KS) void fp8_tiled_kernel(
    const uint8_t *__restrict__ Aall, const float *__restrict__ a_scale,
    const int32_t *__restrict__ a_rows, int M_a, const uint8_t *__restrict__ Wall,
    const float *__restrict__ Sall, const int32_t *__restrict__ offsets, int E, int M, int N,
    int K, int KB, int NB, int nbn, uint16_t *__restrict__ C)
{
    fp8_tile<BM, BN, WM, WN, KS, BF16>(Aall, a_scale, a_rows, M_a, Wall, Sall, offsets, E, M, N, K, KB, NB, 0, nbn, C,
                                       blockIdx.x);
}

// Dense, the first `large` workgroups 256 x 256 tiles of the first nbn column blocks,
// the others BM x BN tiles of the rest, in one launch: a CU that has done its
// large tiles begins with a small one (M x K x N = 4096 x 17408 x 5120: 349 us, as two
// launches 353).
template <int BM, int BN, int WM, int WN, int KS, bool BF16>
__global__ __launch_bounds__(512) void fp8_two_tiles_kernel(
    const uint8_t *__restrict__ Aall, const float *__restrict__ a_scale,
    const int32_t *__restrict__ a_rows, int M_a, const uint8_t *__restrict__ Wall,
    const float *__restrict__ Sall, int M, int N, int K, int KB, int NB, int nbn, int large,
    uint16_t *__restrict__ C)
{
    static_assert(WM * WN * KS == 8, "as many waves as the large tile");
    if ((int)blockIdx.x < large)
        fp8_tile<256, 256, 4, 2, 1, BF16>(Aall, a_scale, a_rows, M_a, Wall, Sall, nullptr, 1, M, N, K, KB, NB, 0, nbn,
                                          C, blockIdx.x);
    else
        fp8_tile<BM, BN, WM, WN, KS, BF16>(Aall, a_scale, a_rows, M_a, Wall, Sall, nullptr, 1, M, N, K, KB, NB,
                                           nbn * 256, (N - nbn * 256 + BN - 1) / BN, C, blockIdx.x - large);
}

// ---- streaming kernel, few rows ----
// For row blocks of 16 MT <= 64 rows the weights are read once.  A workgroup
// holds NT 16-column tiles; its NW waves take the 128-k steps in turn, each with
// a ring of P stages in LDS of its own, so that nothing waits for another wave
// until the partial sums meet, in the order of the waves.  Every load of a
// stage (W tile, A tile, the rows' scales and the weight block's) goes straight
// to LDS: eight lanes read one 128-byte line (loads to the operand registers
// reach 64 bytes of a row at a time and stream at half the rate), and the
// wave's counted wait is exact because it has no other loads.  One row at 5120 x
// 17408: 18.4 us, 4.8 TB/s of weights; 16 tokens to 8 of 64 experts at 2048 x 7168 (830
// MB): 111 to 118 us, 7.3 TB/s.
template <int N>
__device__ inline void wait_loads()
{
    // (a compiler barrier too: the stage's LDS reads stay behind it)
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int MT, int NT, int NW, int P, bool BF16>
__global__ __launch_bounds__(64 * NW) void fp8_stream_kernel(
    const uint8_t *__restrict__ Aall, const float *__restrict__ a_scale,
    const int32_t *__restrict__ a_rows, int M_a, const uint8_t *__restrict__ Wall,
    const float *__restrict__ Sall, const int32_t *__restrict__ offsets, int E, int M, int N,
    int K, int KB, int NB, uint16_t *__restrict__ C)
{
    constexpr int BM = 16 * MT, BN = 16 * NT;
    constexpr int LW = BN / 8, LA = BM / 8, L = LW + LA + 2;     // loads of a stage
    constexpr int STAGE = (BN + BM) * KB8 + 512;                 // tiles, then 64 row scales, then the weight's
    static_assert(MT <= 4 && 128 % BN == 0, "one load for the rows' scales, one weight scale");
    static_assert((P - 1) * L < 64, "vmcnt holds 6 bits");
    static_assert((2 * P - 1) * NW <= MAX_AHEAD, "the scalar offset of the last refill");
    static_assert(MT * NT * 1024 <= P * STAGE, "the partial sums fit in the ring");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int nbn = (N + BN - 1) / BN;
    const int rb = blockIdx.x / nbn, n0 = (blockIdx.x - rb * nbn) * BN;
    RowScan scan = {};
    if (offsets) scan = scan_rows(offsets, E, M, BM, 0);
    const RowBlock blk = find_rows(offsets, E, M, BM, rb, scan);
    const int e = __builtin_amdgcn_readfirstlane(blk.e);
    const int m0 = __builtin_amdgcn_readfirstlane(blk.m0);
    const int m1 = __builtin_amdgcn_readfirstlane(blk.m1);
    if (m0 >= m1) return;      // no such row block: uniform, before the barrier
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int rows_n = N - n0 < BN ? N - n0 : BN, rows_m = m1 - m0 < BM ? m1 - m0 : BM;
    const __amdgpu_buffer_rsrc_t w_rs = buffer_rsrc(Wall + ((size_t)e * N + n0) * K, (size_t)rows_n * K);
    const __amdgpu_buffer_rsrc_t a_rs =
        a_rows ? buffer_rsrc(Aall, (size_t)M_a * K) : buffer_rsrc(Aall + (size_t)m0 * K, (size_t)rows_m * K);
    const __amdgpu_buffer_rsrc_t sa_rs = a_rows ? buffer_rsrc(a_scale, (size_t)M_a * KB * 4)
                                                : buffer_rsrc(a_scale + (size_t)m0 * KB, (size_t)rows_m * KB * 4);
    const __amdgpu_buffer_rsrc_t sw_rs = buffer_rsrc(Sall + ((size_t)e * NB + n0 / 128) * KB, (size_t)KB * 4);

    // row of A that row i of the block takes (the last row again past the end),
    // -1 for an index that names none
    auto row_of = [&](int i) {
        i = m0 + i < m1 ? i : m1 - 1 - m0;
        if (!a_rows) return i;
        const int r = a_rows[m0 + i];
        return (unsigned)r < (unsigned)M_a ? r : -1;
    };
    const int chunk = (lane & 7) ^ (lane >> 3);
    unsigned w_off[LW], a_off[LA];
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        int r = i * 8 + (lane >> 3);
        r = r < rows_n ? r : rows_n - 1;
        w_off[i] = (unsigned)r * (unsigned)K + chunk * 16;
    }
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = row_of(i * 8 + (lane >> 3));
        a_off[i] = (unsigned)(r < 0 ? 0 : r) * (unsigned)K + chunk * 16;
    }
    const int srow = row_of(lane < BM ? lane : 0);
    const unsigned s_off = (unsigned)(srow < 0 ? 0 : srow) * (unsigned)KB * 4u;
    uint8_t *ring = lds + wave * (P * STAGE);

    // (chunks past the end of K, and steps past the last, read nothing and give
    // zeros, scales too)
    auto load = [&](int kt, int sl) {
        uint8_t *base = ring + sl * STAGE;
        const bool in = kt * KB8 + chunk * 16 < K;
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            unsigned off = in ? w_off[i] : FP8_PAST;
            pin(off);
            uint8_t *dst = base + i * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(w_rs, (__attribute__((address_space(3))) void *)dst, 16, off, kt * KB8, 0, QG_NT);
        }
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            unsigned off = in ? a_off[i] : FP8_PAST;
            pin(off);
            uint8_t *dst = base + (LW + i) * 1024;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(a_rs, (__attribute__((address_space(3))) void *)dst, 16, off, kt * KB8, 0, 0);
        }
        unsigned os = kt < KB ? s_off : FP8_PAST, ow = kt < KB ? 0u : FP8_PAST;
        pin(os);
        pin(ow);
        uint8_t *dst = base + (LW + LA) * 1024;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sa_rs, (__attribute__((address_space(3))) void *)dst, 4, os, kt * 4, 0, 0);
        dst += 256;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sw_rs, (__attribute__((address_space(3))) void *)dst, 4, ow, kt * 4, 0, 0);
    };

    float4v acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};
    const int o0 = c * KB8 + ((q ^ (lane & 7)) * 16);
#pragma unroll
    for (int i = 0; i < P; ++i) load(wave + i * NW, i);
    for (int kt = wave; kt < KB; kt += P * NW) {
#pragma unroll
        for (int sl = 0; sl < P; ++sl) {
            // the oldest stage has landed: at most the P - 1 younger ones' loads are in flight
            if (QG_DEBUG_SYNC) wait_loads<0>();
            else wait_loads<(P - 1) * L>();
            const uint8_t *base = ring + sl * STAGE;
            auto operand = [&](int tile) {
                const int4v lo = *reinterpret_cast<const int4v *>(base + tile * 16 * KB8 + o0);
                const int4v hi = *reinterpret_cast<const int4v *>(base + tile * 16 * KB8 + (o0 ^ 64));
                return int8v{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            };
            const float *sc = reinterpret_cast<const float *>(base + (LW + LA) * 1024);
            int8v a[MT], w[NT];
            float s[MT];
#pragma unroll
            for (int j = 0; j < NT; ++j) w[j] = operand(j);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                a[i] = operand(NT + i);
                s[i] = sc[16 * i + c] * sc[64 + lane];
            }
            // the stage is in registers: refill it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            load(kt + (sl + P) * NW, sl);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float4v p = mfma_fp8(w[j], a[i], float4v{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s[i], acc[i][j][r]);
                }
        }
    }
    // the last (empty) loads would write over the partial sums
    wait_loads<0>();
    float4v *part = reinterpret_cast<float4v *>(ring);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[(i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    const bool wide = N % 4 == 0 && ((uintptr_t)C & 7) == 0;
#pragma unroll
    for (int t = 0; t < MT * NT; ++t) {
        if (t % NW != wave) continue;
        const int i = (t / NT) * 16 + c, n = n0 + (t % NT) * 16 + 4 * q;
        float4v x = *(reinterpret_cast<const float4v *>(lds) + t * 64 + lane);
#pragma unroll
        for (int w = 1; w < NW; ++w)
            x += *(reinterpret_cast<const float4v *>(lds + w * (P * STAGE)) + t * 64 + lane);
        if (m0 + i < m1) store4<BF16>(C + (size_t)(m0 + i) * N + n, x, row_of(i) < 0, n, N, wide);
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
long long row_blocks(bool grouped, int E, int M, int BM)
{
    if (!grouped) return (M + BM - 1) / BM;
    return (long long)M / BM + (E < M ? E : M);
}

// The kernel of a call: the streaming ones by their m-tiles, n-tiles and waves,
// the tiled ones by their tile.
enum Fp8Kernel {
    S1x2x4, S1x2x2, S1x1x4, S2x2x4, S2x4x2, S4x2x4, S4x4x4,
    T64x64K2, T64x128, T64x128K2, T128x128K2, T128x256W4, T128x256, T256x256
};

struct Fp8Shape {
    const char *name;
    int bm, bn, threads;
};
constexpr Fp8Shape FP8_SHAPES[] = {
    {"streaming, 16 x 32, 4 waves over k", 16, 32, 256},  {"streaming, 16 x 32, 2 waves over k", 16, 32, 128},
    {"streaming, 16 x 16, 4 waves over k", 16, 16, 256},  {"streaming, 32 x 32, 4 waves over k", 32, 32, 256},
    {"streaming, 32 x 64, 2 waves over k", 32, 64, 128},  {"streaming, 64 x 32, 4 waves over k", 64, 32, 256},
    {"streaming, 64 x 64, 4 waves over k", 64, 64, 256},
    {"tiled, 64 x 64, 2 groups over k", 64, 64, 512},     {"tiled, 64 x 128", 64, 128, 256},
    {"tiled, 64 x 128, 2 groups over k", 64, 128, 512},   {"tiled, 128 x 128, 2 groups over k", 128, 128, 512},
    {"tiled, 128 x 256, 4 waves", 128, 256, 256},         {"tiled, 128 x 256", 128, 256, 512},
    {"tiled, 256 x 256", 256, 256, 512}};

// By the rows an expert has on average (the host does not know the counts; an
// uneven split is slower, never wrong) and the workgroups that makes.  Both
// sides measured in us at K x N = 5120 x 17408 unless stated.
Fp8Kernel choose(bool grouped, int E, int M, int N, int K)
{
    const long long active = grouped ? (E < M ? E : M) : 1;
    const long long rows = (M + active - 1) / active;
    auto wgs = [&](int bm, int bn) { return active * ((rows + bm - 1) / bm) * ((N + bn - 1) / bn); };
    if (rows <= 16) {
        // enough workgroups that a smaller share of K each pays: 16 tokens to 8 of
        // 64 experts at 2048 x 7168: 114 (two waves) against 129 (four)
        if (wgs(16, 32) >= 2048) return S1x2x2;
        // too few for the chip and a short K: four rows at 2048 x 2048: 3.9
        // (16 columns) against 4.4 (32); at 17408 x 5120 28.5 against 22.5
        if (wgs(16, 32) < 128 && K <= 4096) return S1x1x4;
        return S1x2x4;                                   // one row: 18.8, tiled 43.9
    }
    // 32 rows: 27.2, as two blocks of 16 35.0, tiled 44.4; 16 rows an
    // expert in 64 experts at 2048 x 7168: 174 (32 x 64) against 225 (32 x 32)
    if (rows <= 32) return wgs(32, 32) >= 2048 ? S2x4x2 : S2x2x4;
    const long long w64 = wgs(64, 128), w128 = wgs(128, 128), w256 = wgs(256, 256);
    if (rows <= 128 && w64 <= 128) {
        // Few tiles: the streaming kernels make more workgroups.  64 rows at 17408 x
        // 5120: 42.8, 64 x 64 tiles 63.7; 128 rows there: 55 (64 columns), 62; 100 rows at
        // 640 x 1000: 4.6, tiled 5.0
        if (rows <= 64 || K <= 4096) return S4x2x4;
        return S4x4x4;
    }
    if (rows > 128) {
        // 512 rows (136 large tiles): 71 against 94 for 64 x 128 and 101 for 128 x 256; 256
        // rows (136 tiles of 128 x 256): 58 against 64 (64 x 128) and 73 (68 large tiles);
        // 2000 rows at 4096 x 4096 (256 or 128): 44 against 52
        const long long w = wgs(128, 256);
        if (w256 >= 192 || (w256 >= 128 && w > 256)) return T256x256;
        // four waves read less from LDS, eight wait less: 1024 rows at 8192 columns, K = 2048
        // 23.9 and 22.9, 5120 56 and 58; 256 at 17408 columns, K = 2048 22.7 and 20.9
        if (w > 128 && w <= 256) return K <= 4096 ? T128x256 : T128x256W4;
    }
    // 65 to 128 rows and many tiles: the large tile reads the weights once, and its waves
    // without rows cost little.  100 rows at 5120 x 50257 (197 tiles): 81 us against 104
    // (64 x 128); 100 an expert in 8 at 2048 x 7168 (224): 33 against 45, in 64: 262
    // against 290.  Not where 64 x 128 is one round (three to a CU; 85 in 8 at 4096 x 6144:
    // 63 against 56), large tiles leave over a quarter of their rounds empty (93 in 30 at
    // 2048 x 3000: 63 against 59), K is short (70 in 60 at 1024 x 2048: 41 against 37) or,
    // in several rounds, rows are few (75 in 32 at 2048 x 7168: 123 against 120).
    const long long rounds = (w256 + 255) / 256;
    if (K >= 2048 && w64 > 768 && w256 * 4 >= rounds * 256 * 3 && rows > (rounds == 1 ? 64 : 80)) return T256x256;
    // One tile to a CU at most: two groups over k.  256 rows at 4096 x 8192 (256 tiles):
    // 18.6 against 22.3; 64 rows (136): 34.4, 40.7, streaming 39.8; 300 rows at 2000 x
    // 3000 (235 tiles of 64 x 64): 10 against 14
    if (w64 <= 128) return T64x64K2;
    if (w64 <= 256) return T64x128K2;
    // 128 rows (136 tiles): 40 against 48; 512 rows at 17408 x 5120 (160): 107, 135
    if (rows > 64 && w128 <= 256) return T128x128K2;
    // (up to 128 rows an expert, many tiles)
    return T64x128;
}

template <int BM, int BN, int WM, int WN, int KS>
constexpr int tile_lds() { return KS * (2 * (BM + BN) * KB8 + WM * WN * (BM / WM / 16) * 256) + BM * 4; }

hipError_t allow_lds(const void *kern, int bytes)
{
    if (bytes <= 65536) return hipSuccess;
    return hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int BM, int BN, int WM, int WN, int KS, bool BF16>
hipError_t tiled(const Fp8Args &a, hipStream_t st)
{
    const auto kern = fp8_tiled_kernel<BM, BN, WM, WN, KS, BF16>;
    constexpr int bytes = tile_lds<BM, BN, WM, WN, KS>();
    const hipError_t e = allow_lds((const void *)kern, bytes);
    if (e != hipSuccess) return e;
    const int nbn = (a.N + BN - 1) / BN;
    const long long wgs = row_blocks(a.offsets != nullptr, a.E, a.M, BM) * nbn;
    hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(64 * WM * WN * KS), bytes, st, a.A, a.a_scale, a.a_rows,
                       a.M_a, a.W, a.w_scale, a.offsets, a.E, a.M, a.N, a.K, a.KB, a.NB, nbn, a.C);
    return hipGetLastError();
}

// The large tile on the first nbn column blocks, a small one on the rest.
template <int BM, int BN, int WM, int WN, int KS, bool BF16>
hipError_t two_tiles(const Fp8Args &a, int nbn, hipStream_t st)
{
    const auto kern = fp8_two_tiles_kernel<BM, BN, WM, WN, KS, BF16>;
    constexpr int large_lds = tile_lds<256, 256, 4, 2, 1>(), small_lds = tile_lds<BM, BN, WM, WN, KS>();
    constexpr int bytes = large_lds > small_lds ? large_lds : small_lds;
    const hipError_t e = allow_lds((const void *)kern, bytes);
    if (e != hipSuccess) return e;
    const int large = (a.M + 255) / 256 * nbn;
    const int small = (a.M + BM - 1) / BM * ((a.N - nbn * 256 + BN - 1) / BN);
    hipLaunchKernelGGL(kern, dim3(large + small), dim3(512), bytes, st, a.A, a.a_scale, a.a_rows, a.M_a, a.W,
                       a.w_scale, a.M, a.N, a.K, a.KB, a.NB, nbn, large, a.C);
    return hipGetLastError();
}

// The large tile.  Where its grid is some rounds of the chip's 256 CUs and part of one, the
// column blocks past the whole rounds go to the smallest tile that makes one
// round of them (the counts must be the host's, so not grouped).  us at M = 2048,
// K = 4096, by the tiles past a round of large ones:
//   past     all large   64 x 128   128 x 128   128 x 256
//     16        108          81          85          97
//     48        112         101          90         104
//     88        120         129         120         113
//    152        126                                 147
struct LargeSplit {
    int nbn;             // column blocks of large tiles, 0 for all of them
    Fp8Kernel rest;      // the tile of the other columns
};

LargeSplit large_split(bool grouped, int M, int N)
{
    const long long rbs = (M + 255) / 256, tiles = rbs * ((N + 255) / 256);
    const int nbn = (int)(tiles / 256 * 256 / rbs);
    const long long cols = N - (long long)nbn * 256;
    if (grouped || nbn == 0 || cols <= 0) return {0, T256x256};
    for (const Fp8Kernel rest : {T64x128K2, T128x128K2, T128x256}) {
        const Fp8Shape &k = FP8_SHAPES[rest];
        if (((M + k.bm - 1) / k.bm) * ((cols + k.bn - 1) / k.bn) <= 256) return {nbn, rest};
    }
    return {0, T256x256};
}

template <bool BF16>
hipError_t large_tiles(const Fp8Args &a, hipStream_t st)
{
    const LargeSplit x = large_split(a.offsets != nullptr, a.M, a.N);
    if (x.nbn == 0) return tiled<256, 256, 4, 2, 1, BF16>(a, st);
    if (x.rest == T64x128K2) return two_tiles<64, 128, 2, 2, 2, BF16>(a, x.nbn, st);
    if (x.rest == T128x128K2) return two_tiles<128, 128, 2, 2, 2, BF16>(a, x.nbn, st);
    return two_tiles<128, 256, 2, 4, 1, BF16>(a, x.nbn, st);
}

template <int MT, int NT, int NW, int P, bool BF16>
hipError_t stream(const Fp8Args &a, hipStream_t st)
{
    const auto kern = fp8_stream_kernel<MT, NT, NW, P, BF16>;
    constexpr int bytes = NW * P * (16 * (MT + NT) * KB8 + 512);
    const hipError_t e = allow_lds((const void *)kern, bytes);
    if (e != hipSuccess) return e;
    const long long wgs = row_blocks(a.offsets != nullptr, a.E, a.M, 16 * MT) * ((a.N + 16 * NT - 1) / (16 * NT));
    hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(64 * NW), bytes, st, a.A, a.a_scale, a.a_rows, a.M_a, a.W,
                       a.w_scale, a.offsets, a.E, a.M, a.N, a.K, a.KB, a.NB, a.C);
    return hipGetLastError();
}

template <bool BF16>
hipError_t launch(const Fp8Args &a, hipStream_t st)
{
    switch (choose(a.offsets != nullptr, a.E, a.M, a.N, a.K)) {
    case S1x2x4: return stream<1, 2, 4, 2, BF16>(a, st);
    case S1x2x2: return stream<1, 2, 2, 2, BF16>(a, st);
    case S1x1x4: return stream<1, 1, 4, 2, BF16>(a, st);
    case S2x2x4: return stream<2, 2, 4, 2, BF16>(a, st);
    case S2x4x2: return stream<2, 4, 2, 2, BF16>(a, st);
    case S4x2x4: return stream<4, 2, 4, 2, BF16>(a, st);
    case S4x4x4: return stream<4, 4, 4, 2, BF16>(a, st);
    case T64x64K2: return tiled<64, 64, 2, 2, 2, BF16>(a, st);
    case T64x128: return tiled<64, 128, 2, 2, 1, BF16>(a, st);
    case T64x128K2: return tiled<64, 128, 2, 2, 2, BF16>(a, st);
    case T128x128K2: return tiled<128, 128, 2, 2, 2, BF16>(a, st);
    case T128x256W4: return tiled<128, 256, 2, 2, 1, BF16>(a, st);
    case T128x256: return tiled<128, 256, 2, 4, 1, BF16>(a, st);
    case T256x256: return large_tiles<BF16>(a, st);
    }
    return hipErrorUnknown;
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

long long fp8_threads(bool grouped, int E, int M, int N, int K)
{
    const Fp8Shape &k = FP8_SHAPES[choose(grouped, E, M, N, K)];
    return row_blocks(grouped, E, M, k.bm) * ((N + k.bn - 1) / k.bn) * k.threads;
}

void describe_fp8(bool grouped, int E, int M, int N, int K, char *buf, size_t n)
{
    const Fp8Kernel kern = choose(grouped, E, M, N, K);
    const LargeSplit x = kern == T256x256 ? large_split(grouped, M, N) : LargeSplit{0, kern};
    if (x.nbn)
        snprintf(buf, n, "%s, from column %d on %s", FP8_SHAPES[kern].name, x.nbn * 256,
                 FP8_SHAPES[x.rest].name + strlen("tiled, "));
    else
        snprintf(buf, n, "%s", FP8_SHAPES[kern].name);
}

} // namespace qg
