// Ragged batches: runs of rows whose counts stand in device memory (gfx950 only).
#pragma once

#include "qg_device.h"

namespace qg {

// n rows from `row` on; len: what else a run's count depends on.
struct Run {
    int row, n, len;
};

// Rows off[b] .. off[b + 1] - 1, kept inside 0 .. T - 1 whatever stands there.
__device__ inline Run run_of(const int32_t *__restrict__ off, int T, int b)
{
    int r0 = off[b], r1 = off[b + 1];
    r0 = r0 < 0 ? 0 : (r0 > T ? T : r0);
    r1 = r1 < r0 ? r0 : (r1 > T ? T : r1);
    return Run{r0, r1 - r0, 0};
}

// The sum of the values of a lane and of those before it: in each row of 16 lanes, then the
// rows' last values on to the rows behind.
__device__ inline int scan64(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);      // from 1, 2, 4, 8 lanes before
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);      // lane 15 to row 1, lane 47 to row 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);      // lane 31 to rows 2 and 3
    return v;
}

// Item x of all runs' items, count(run) of each that has rows, in order: its run b, its
// place `in` there out of `of`.  The grid is an upper bound and every wave scans the
// counts for itself, 64 runs a step (run(b) for a lane's b, also past the last: no rows).
// False if there are fewer items.
template <class G, class F>
__device__ inline bool find_item(int B, int x, G run, F count, int &b, int &in, int &of, Run &got)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        const Run q = run(b0 + lane);
        const int mine = q.n > 0 ? count(q) : 0;
        const int sum = scan64(mine);
        const unsigned long long hit = __ballot(base + sum > x);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            b = b0 + l;
            of = __builtin_amdgcn_readlane(mine, l);
            in = x - (base + __builtin_amdgcn_readlane(sum, l) - of);
            got.row = __builtin_amdgcn_readlane(q.row, l);
            got.n = __builtin_amdgcn_readlane(q.n, l);
            got.len = __builtin_amdgcn_readlane(q.len, l);
            return true;
        }
        base += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

} // namespace qg
