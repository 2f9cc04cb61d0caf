// ds_tree.cuh -- what the tree-attention kernels share: arguments, the split of
// the work over CTAs and the layout of partial results.
//
// Work. The t * G query rows of one (entry, kv head) (row r is node r / G, head
// r % G of the group) form row tiles; the rows of the cache form token tiles.
// A row tile against all token tiles of its entry is an item, numbered
// (entry, kv head, row tile); a unit is one token tile of an item. The units
// of all items, in order, are dealt to the CTAs in equal consecutive shares,
// whatever the entries' lengths are (they are known on the device only). A
// CTA that holds all units of an item writes its output; a shorter piece
// leaves its rows' running maximum, sum and weighted values in the workspace,
// and the combine kernel joins an item's pieces.
#pragma once

#include "ds_common.cuh"
#include "ds_internal.h"

namespace ds {

struct TreeParams {
    const void *q, *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *mask, *seq_lens, *node_lens;
    CacheRows at;
    int b, t, hq, hkv, G, s;
    long long cache_rows;  // rows of the whole cache or pool
    int rows;        // t * G
    int tile_rows;   // rows of a row tile
    int n_mt;        // row tiles of a (entry, kv head)
    int tile_tokens; // tokens of a token tile
    int grid;        // CTAs of the attention launch
    float qscale;    // sm_scale * log2(e)
    void* out;
    int out_bf16;
    float* part;     // partial results: see part_of
    float* sums;     // second accumulators of ds_tree_tc.cu, where pieces may be long; or NULL
    int part_rows;   // rows of a partial: min(rows, tile_rows), rounded up to a multiple of 4
    unsigned int* err;
};

// Prefix and node counts of entry e.
__device__ __forceinline__ int tree_prefix(const TreeParams& p, int e) {
    return p.seq_lens ? min(max(__ldg(p.seq_lens + e), 0), p.s) : p.s;
}
__device__ __forceinline__ int tree_nodes(const TreeParams& p, int e) {
    return p.node_lens ? min(max(__ldg(p.node_lens + e), 0), p.t) : p.t;
}
// Units of an entry's items together, and of one item.
__device__ __forceinline__ int item_units(const TreeParams& p, int e) {
    const int n = tree_nodes(p, e);
    return n > 0 ? (tree_prefix(p, e) + n + p.tile_tokens - 1) / p.tile_tokens : 0;
}

// Units before entry e (called by whole warps).
__device__ __forceinline__ long long tree_before(const TreeParams& p, int e) {
    const long long per = (long long)p.hkv * p.n_mt;
    if (!p.seq_lens && !p.node_lens) return (long long)item_units(p, 0) * per * e;
    long long sum = 0;
    for (int x = lane_id(); x < e; x += 32) sum += item_units(p, x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum * per;
}

// A place in the order of units. Every member is the same in all lanes.
struct TreeCursor {
    int e = 0;                // entry
    long long base = 0;       // units before the entry
    int units = 0;            // units of one item of the entry
    int prefix = 0, nodes = 0;
};

__device__ __forceinline__ void cursor_entry(const TreeParams& p, TreeCursor& c, int e) {
    c.e = e;
    c.prefix = tree_prefix(p, e);
    c.nodes = tree_nodes(p, e);
    c.units = c.nodes > 0 ? (c.prefix + c.nodes + p.tile_tokens - 1) / p.tile_tokens : 0;
}

// Units of the whole call (called by whole warps).
__device__ __forceinline__ long long tree_total(const TreeParams& p) { return tree_before(p, p.b); }

// The cursor whose entry holds unit u < total (called by whole warps).
__device__ __forceinline__ TreeCursor tree_seek(const TreeParams& p, long long u) {
    const long long per = (long long)p.hkv * p.n_mt;
    TreeCursor c;
    if (!p.seq_lens && !p.node_lens) {
        const long long n = (long long)item_units(p, 0) * per;
        const int e = (int)((u | n) >> 31 ? u / n : (long long)((unsigned)u / (unsigned)n));
        c.base = (long long)e * n;
        cursor_entry(p, c, e);
        return c;
    }
    long long base = 0;
    for (int e0 = 0; e0 < p.b; e0 += 32) {
        const int e = e0 + lane_id();
        const long long n = e < p.b ? item_units(p, e) * per : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane_id() >= o) incl += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > u);
        if (past) {
            const int l = __ffs(past) - 1;
            c.base = base + __shfl_sync(0xffffffffu, incl - n, l);
            cursor_entry(p, c, e0 + l);
            return c;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    cursor_entry(p, c, p.b - 1);  // not reached for u < total
    c.base = base - c.units * per;
    return c;
}

// The shares of `grid` CTAs of `total` units: the first `extra` have one more
// than the others' `each`.
struct TreeShares {
    long long each;
    int extra;
    __device__ __forceinline__ TreeShares(long long total, int grid) {
        if (total >> 31) {
            each = total / grid;
            extra = (int)(total - each * grid);
        } else {
            const unsigned q = (unsigned)total / (unsigned)grid;
            each = q;
            extra = (int)((unsigned)total - q * (unsigned)grid);
        }
    }
    // First unit of CTA i's share (share i ends where share i + 1 begins).
    __device__ __forceinline__ long long begin(int i) const { return each * i + min(i, extra); }
    // The CTA whose share holds unit u.
    __device__ __forceinline__ int holder(long long u) const {
        const long long wide = (each + 1) * extra;
        if (u < wide) return (int)quotient(u, each + 1);
        return extra + (int)quotient(u - wide, each);
    }
    static __device__ __forceinline__ long long quotient(long long a, long long b) {
        return (a | b) >> 31 ? a / b : (long long)((unsigned)a / (unsigned)b);
    }
};

// A CTA's piece of one item.
struct TreePiece {
    int e, h, mt;          // entry, kv head, row tile
    int prefix, nodes;
    int t0, t1;            // token tiles [t0, t1) of the item's `units`
    int units;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == units; }
};

// The pieces of share [u, end), one by one; false when there is none left.
__device__ __forceinline__ bool next_piece(const TreeParams& p, TreeCursor& c, long long& u, long long end,
                                           TreePiece& w) {
    if (u >= end) return false;
    const int per = p.hkv * p.n_mt;
    while (u >= c.base + (long long)c.units * per) {
        c.base += (long long)c.units * per;
        cursor_entry(p, c, c.e + 1);
    }
    const long long in_entry = u - c.base;
    const int item = (int)TreeShares::quotient(in_entry, c.units);
    w.e = c.e; w.h = item / p.n_mt; w.mt = item - w.h * p.n_mt;
    w.prefix = c.prefix; w.nodes = c.nodes; w.units = c.units;
    w.t0 = (int)(in_entry - (long long)item * c.units);
    const long long left = end - u;
    w.t1 = left < c.units - w.t0 ? w.t0 + (int)left : c.units;
    u += w.t1 - w.t0;
    return true;
}

// Partial results. CTA i has two places: 1 for a piece that begins its item, 0
// for one that continues it (a share holds at most one unfinished piece of
// each kind). A place holds, for each of part_rows rows, the running maximum
// (of score * log2 e), the sum, and then the weighted values [part_rows][D].
__device__ __forceinline__ float* part_of(const TreeParams& p, int cta, int begins, int d) {
    return p.part + ((size_t)cta * 2 + begins) * ((size_t)p.part_rows * (d + 2));
}

// Element offset of query row `row` of (entry, kv head) in q and out.
__device__ __forceinline__ size_t q_offset(const TreeParams& p, int e, int h, int row, int d) {
    const int node = row / p.G, g = row - node * p.G;
    return (((size_t)e * p.t + node) * p.hq + (size_t)h * p.G + g) * d;
}
// Word w of the mask row of (entry e, node i): which nodes 32w .. it sees.
__device__ __forceinline__ uint32_t mask_word(const TreeParams& p, int e, int i, int w) {
    if (p.mask) {
        const int words = (p.t + 31) / 32;
        return (uint32_t)__ldg(p.mask + ((size_t)e * p.t + i) * words + w);
    }
    const int n = i + 1 - 32 * w;  // a chain: nodes 0 .. i
    return n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
}
// Pool or cache row of token t for reading; block ids are clamped.
__device__ __forceinline__ long long tree_row(const CacheRows& c, int e, int h, int t) {
    if (!c.block_table) return ((long long)e * c.hkv + h) * c.s_cap + t;
    int blk = __ldg(c.block_table + (size_t)e * c.max_blocks + (t >> c.page_shift));
    blk = min(max(blk, 0), c.num_blocks - 1);
    return (((long long)blk * c.hkv + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

// Token tiles of a stream between two moves of its tensor-core sums (ds_tree_tc.cuh).
constexpr int kTreeSpan = 128;

enum TreeType { kTreeF32 = 0, kTreeBF16 = 1, kTreeE4M3 = 2 };

// Launches. f32 (ds_tree_simt.cu):
struct TreePlan { int tile_rows, tile_tokens, grid; };
TreePlan plan_tree_simt(int rows, int d);
cudaError_t launch_tree_simt(const TreeParams& p, int d, cudaStream_t st);
// bf16 and e4m3 (ds_tree_tc.cu; up to 16 query rows, e4m3 32: ds_tree_few.cu).
TreePlan plan_tree_tc(int rows, int type);
// Bytes of their second accumulators, for pieces of at most `tiles` token tiles.
size_t tree_tc_sums(const TreePlan& plan, int grid, long long tiles, int d);
cudaError_t launch_tree_tc(const TreeParams& p, int type, int d, cudaStream_t st);
cudaError_t launch_tree_combine(const TreeParams& p, int d, cudaStream_t st);

}  // namespace ds
