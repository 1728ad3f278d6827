// The paged 4-bit key/value cache as the kernels see it (gfx950 only).
//
// A token's row of D channels of one head is D/g groups of g channels; each holds
// 4-bit codes, an fp16 scale s and an fp16 zero z, and stands for code * s + z.
//
// Codes are laid out as operands of the 16x16x32 fp16 MFMA, made without a
// multiplication or an exchange between lanes: two nibbles of a word, shifted to bits 4 to 7 of
// its halves and ORed with the exponent of 64, are the binary16 values 64 + code, and
// 64 times the sum of the other operand is taken off the product again.
//   keys    a token's D/8 words are [4][D/32]: lane group q of the MFMA owns words
//           (q, 0 .. D/32 - 1).  Nibble 4a + 2b + c of word (q, 2i + l) is channel
//           32 (i + c D/64) + 8 q + 4 l + 2 b + a: words 2i, 2i + 1 hold the eight
//           channels of k-step i in their low and of step i + D/64 in their high
//           nibbles.
//   values  the words of 32 consecutive tokens are [D/64][4][16][4]: one 16-byte load
//           gives lane (q, m) words j = 0 .. 3, and nibble 4a + 2b + c of word (u, q, m,
//           j) is channel 64 u + 16 j + m of token 16 c + 4 q + 2 b + a: the eight
//           tokens whose probabilities the same lane holds after the products with two
//           16-token tiles of keys, so these need no exchange between lanes.
// Both take D/8 words a token, so a 32-token block of a head starts at the same
// offset in either.  Scale and zero of a group are one word (scale low), [page][head]
// [D/g][page_size].
#pragma once

#include "qg_ragged.h"

namespace qg {

constexpr int KV4_BLOCK = 32;      // tokens that share words

struct Kv4Cache {
    uint32_t *k, *v, *k_sz, *v_sz;
    int pages, heads, shift;       // page_size == 1 << shift, shift >= 5
    int D, g;
};

struct Kv4Batch {
    const int32_t *off, *lens, *table;   // off: nullptr, or [B + 1] row offsets
    int B, width, T;                     // width: page table entries of a sequence
};

// The rows of sequence b: n of them, the last ones of its len tokens.
__device__ inline Run kv4_seq(const Kv4Batch &s, int b)
{
    if (b >= s.B) return Run{0, 0, 0};
    Run q = s.off ? run_of(s.off, s.T, b) : Run{b, 1, 0};
    const int len = s.lens[b];
    q.len = len < 0 ? 0 : len;
    return q;
}

// Item x of all sequences' items, count(seq) of each (ragged batches: find_item).
template <class F>
__device__ inline bool kv4_find(const Kv4Batch &s, int x, F count, int &b, int &in, int &of, Run &seq)
{
    if (s.off) return find_item(s.B, x, [&](int i) { return kv4_seq(s, i); }, count, b, in, of, seq);
    of = count(Run{0, 1, 1});          // one row each: the same count for all
    b = x / of;
    in = x - b * of;
    if (b >= s.B) return false;
    seq = kv4_seq(s, b);
    return true;
}

// The 32-token blocks that a sequence's new rows lie in (their indices may begin
// below zero: rows without a place in the cache).
__device__ inline int kv4_row_blocks(const Run &q)
{
    return ((q.len - 1) >> 5) - ((q.len - q.n) >> 5) + 1;
}
// At most this many for all: n rows lie in at most n / 32 + 2 blocks, and in n.
inline long long kv4_row_blocks_bound(int T, int B)
{
    const long long n = T / KV4_BLOCK + 2ll * B;
    return n < T ? n : T;
}

// The page of a token of sequence b, -1 if the table names none.
__device__ inline int kv4_page(const Kv4Cache &c, const Kv4Batch &s, int b, int t)
{
    const int i = t >> c.shift;
    if (t < 0 || i >= s.width) return -1;
    const int p = s.table[(size_t)b * s.width + i];
    return (unsigned)p < (unsigned)c.pages ? p : -1;
}

} // namespace qg
