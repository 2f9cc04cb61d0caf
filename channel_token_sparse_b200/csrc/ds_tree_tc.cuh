// ds_tree_tc.cuh -- what the tensor-core kernels of the tree attention share:
// tcgen05 wrappers, bounded waits, the ring of K and V stages and its loaders.
#pragma once

#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kT = 128;  // tokens of a tile, and rows of a row block

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_ld(uint32_t (&r)[8], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                   : "memory");
}
__device__ __forceinline__ void tc_ld(uint32_t (&r)[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
                 "%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                 "%12,%13,%14,%15,%16};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) :
                   "memory");
}
__device__ __forceinline__ void tc_ld(uint32_t (&r)[32], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
                 "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,"
                 "%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                   "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                   "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) :
                   "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets (in 16-byte units), version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)(addr >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: bf16 x bf16 -> f32, M = 128, N = n; A and B K-major,
// or (transposed) M- and N-major.
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool a_m_major, bool b_n_major) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_m_major ? 1u << 15 : 0u) | (b_n_major ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
// To N registers from the FROM that the kernel was launched with.
template <int N, int FROM> __device__ __forceinline__ void reg_dec_or_inc() {
    if constexpr (N < FROM) reg_dec<N>();
    else if constexpr (N > FROM) reg_inc<N>();
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------------- waiting

// A wait gives up after about a second, or when another one of the CTA did:
// every role then leaves its loop (see mbar_wait_bounded).
struct Waiter {
    volatile int* stop;
    unsigned int* err;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        return mbar_try_wait(bar, parity) || poll(bar, parity);
    }
    __device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity) const {
        const uint64_t t0 = global_ns();
        for (;;) {
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*stop) return false;
            if (global_ns() - t0 > 1000000000ull) break;
        }
        *stop = 1;
        note_timeout(err, 3);
        return false;
    }
};

// A place in the ring of stages: consecutive uses of stage `i`, phase `ph`.
template <int N> struct Ring {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() { if (++i == N) { i = 0; ph ^= 1; } }
};

// 16 bytes from global to shared memory, or 16 zero bytes (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0));
}

// Byte offset of 16-byte chunk c (eight channels) of row r in a tile: blocks
// of 64 channels of all `rows` rows, 128 bytes a row, chunks exchanged within
// groups of 8 rows.
__device__ __forceinline__ int tile_at(int r, int c, int rows = kT) {
    return (c >> 3) * (rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Visible columns 32w .. 32w + 31 of a token tile for node `node`: c0 is the
// node index of the first of them (negative: prefix), n the number of nodes.
__device__ __forceinline__ uint32_t visible(const TreeParams& p, int e, int node, int n, int c0) {
    if (c0 <= -32) return 0xffffffffu;
    auto word = [&](int w) -> uint32_t {  // which nodes 32w .. the node sees
        const int have = n - 32 * w;
        if (have <= 0) return 0u;
        return mask_word(p, e, node, w) & (have >= 32 ? 0xffffffffu : (1u << have) - 1u);
    };
    if (c0 < 0) return word(0) << -c0 | ((1u << -c0) - 1u);
    const int w = c0 >> 5, sh = c0 & 31;
    return sh ? word(w) >> sh | word(w + 1) << (32 - sh) : word(w);
}

struct RingUse { int i; bool is_v; };  // token tile, of V or K

// Four e4m3 codes -> four bf16 values (exact). A code's sign, exponent and
// mantissa bits at their places in a bf16 are its value times 2^-120 (the
// difference of the exponents' biases, subnormals too); the product with 2^120
// is exact. (The conversion instructions bounded 8-bit tiles.) The NaN code
// becomes +-480: rows that are not finite are marked by their scale.
__device__ __forceinline__ uint32_t widen2(uint32_t x) {  // codes in the halves' high bytes
    uint32_t r = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0x7b807b80u));
    return r;
}
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    return make_uint2(widen2(__byte_perm(w, 0, 0x1404)), widen2(__byte_perm(w, 0, 0x3424)));
}

// The pages of a token tile: a lane keeps the block of the tile's rows 4 lane
// .. 4 lane + 3, so one table read a warp and tile serves its 128 rows. Pages
// of one or two rows are looked up row by row.
struct TilePages {
    int blk = 0;
    __device__ __forceinline__ void load(const CacheRows& c, int e, int tok0, int tokens) {
        if (c.page_shift < 2) return;
        const int t = min(tok0 + 4 * lane_id(), tokens - 1);
        blk = __ldg(c.block_table + (size_t)e * c.max_blocks + (t >> c.page_shift));
        blk = min(max(blk, 0), c.num_blocks - 1);
    }
    // Pool row of token t = tok0 + r < tokens (called by whole warps).
    __device__ __forceinline__ long long row(const CacheRows& c, int e, int h, int t, int r) const {
        if (c.page_shift < 2) return tree_row(c, e, h, t);
        const int b = __shfl_sync(0xffffffffu, blk, r >> 2);
        return (((long long)b * c.hkv + h) << c.page_shift) + (t & ((1 << c.page_shift) - 1));
    }
};

// V columns of fp32 values, waited for.
template <int V> __device__ __forceinline__ void load_columns(float (&x)[V], uint32_t addr) {
    uint32_t y[V];
    tc_ld(y, addr);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __uint_as_float(y[i]);
}
template <int V> __device__ __forceinline__ void store_columns(uint32_t addr, const float (&x)[V]) {
    uint32_t y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = __float_as_uint(x[i]);
    tc_st(addr, y);
}

// Zeroes the values that are not finite in rows [b, b + cnt) of a V stage (the
// tile's tree rows; row 0 is node `node0`, negative in the prefix) and marks
// their nodes; thread t of 128. True where this thread changed something.
template <int D>
__device__ __forceinline__ bool clear_not_finite(uint8_t* v, int b, int cnt, int node0, uint32_t* bad, int t) {
    constexpr int kChunks = D / 8;
    bool changed = false;
    for (int x = t; x < cnt * kChunks; x += 128) {
        const int r = b + x / kChunks;
        uint32_t* at = reinterpret_cast<uint32_t*>(v + tile_at(r, x % kChunks));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t y = at[k];
            const bool lo = (y & 0x7f80u) == 0x7f80u, hi = (y & 0x7f800000u) == 0x7f800000u;
            if (lo || hi) {
                at[k] = y & (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
                atomicOr(bad + ((node0 + r) >> 5), 1u << ((node0 + r) & 31));
                changed = true;
            }
        }
    }
    return changed;
}
// What the marked nodes that `node` sees add to channel c: the sum of their
// values that are not finite (8-bit: NaN, for a row whose scales are not).
template <int TYPE, int D>
__device__ __forceinline__ float not_finite_seen(const TreeParams& p, const TreePiece& w, int node, const uint32_t* bad, int c) {
    float sum = 0.f;
    for (int q = 0; q < 8; ++q) {
        if (!bad[q]) continue;
        for (uint32_t see = bad[q] & mask_word(p, w.e, node, q); see; see &= see - 1) {
            const long long row = tree_row(p.at, w.e, w.h, w.prefix + 32 * q + __ffs(see) - 1);
            if constexpr (TYPE == kTreeE4M3) {
                if (!isfinite(p.k_scale[row] * p.qscale) || !isfinite(p.v_scale[row])) sum = NAN;
            } else {
                const float f = Elem<bf16_t>::to_f32(static_cast<const bf16_t*>(p.v)[row * D + c]);
                if (!isfinite(f)) sum += f;
            }
        }
    }
    return sum;
}

// Adds to a stored result of this thread (element `at` of out, or of a partial).
__device__ __forceinline__ void add_result(const TreeParams& p, float* part, size_t at, float f) {
    if (f == 0.f) return;
    if (part) part[at] += f;
    else if (p.out_bf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
        *o = __float2bfloat16_rn(__bfloat162float(*o) + f);
    } else {
        static_cast<float*>(p.out)[at] += f;
    }
}

// What a CTA's roles share of its shared memory.
struct TcRing {
    uint8_t *q, *stages;             // queries; K and V tiles
    uint64_t *full, *empty, *q_empty;
};

// The queries of a piece: QR rows (in blocks of at most 128), zeros past its own.
template <int D, int QR, int THREADS>
__device__ __forceinline__ void load_queries(const TreeParams& p, const TreePiece& w, uint8_t* q, int tid, bool async) {
    constexpr int kChunks = D / 8, kB = QR < kT ? QR : kT;
    const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
#pragma unroll 2
    for (int x = tid; x < QR * kChunks; x += THREADS) {
        const int row = x / kChunks, c = x % kChunks;
        const bool there = row < rows;
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + (there ? q_offset(p, w.e, w.h, row0 + row, D) : 0) + c * 8;
        uint8_t* dst = q + (row / kB) * kB * D * 2 + tile_at(row % kB, c, kB);
        if (async) copy16(smem_u32(dst), src, there);
        else *reinterpret_cast<uint4*>(dst) = there ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
    }
}

// Loader warps of bf16 caches (128 threads): 16-byte asynchronous copies that
// arrive on the stage's barrier when they land.
template <int D, int NS, int QR, typename Order>
__device__ __forceinline__ void load_bf16(const TreeParams& p, const TcRing& m, const Waiter& wait, TreeCursor cur,
                                          long long u, long long end, int tid) {
    constexpr int kChunks = D / 8, kStep = 128 / kChunks;  // rows the threads cover at a time
    const int c = tid % kChunks, r0 = tid / kChunks;
    Ring<NS> ring;
    uint32_t q_ph = 1;  // the first wait on q_empty passes
    TreePiece w;
    while (next_piece(p, cur, u, end, w)) {
        if (w.nodes * p.G - w.mt * p.tile_rows <= 0) continue;
        const int n = w.t1 - w.t0, tokens = w.prefix + w.nodes;
        if (!__all_sync(0xffffffffu, wait(m.q_empty, q_ph))) break;
        q_ph ^= 1;
        load_queries<D, QR, 128>(p, w, m.q, tid, true);  // they land with the first K tile
        bool ok = true;
        TilePages pages;
        if (p.at.block_table) pages.load(p.at, w.e, w.t0 * kT, tokens);
        for (int k = 0; k < 2 * n; ++k) {
            const RingUse use = Order::use(k, n);
            ok = __all_sync(0xffffffffu, wait(m.empty + ring.i, ring.ph ^ 1));
            if (!ok) break;
            const uint32_t dst = smem_u32(m.stages + ring.i * (kT * D * 2));
            const uint16_t* src = static_cast<const uint16_t*>(use.is_v ? p.v : p.k) + c * 8;
            const int tok0 = (w.t0 + use.i) * kT;
            if (!p.at.block_table) {
                // one run of rows: constant steps from the first
                src += (((long long)w.e * p.at.hkv + w.h) * p.at.s_cap + tok0 + r0) * D;
#pragma unroll
                for (int x = 0; x < kChunks; ++x)
                    copy16(dst + tile_at(r0 + x * kStep, c), src + x * kStep * D, tok0 + r0 + x * kStep < tokens);
            } else {
#pragma unroll 8
                for (int x = 0; x < kChunks; ++x) {
                    const int r = r0 + x * kStep, t = min(tok0 + r, tokens - 1);
                    const long long row = pages.row(p.at, w.e, w.h, t, r);
                    copy16(dst + tile_at(r, c), src + row * D, tok0 + r < tokens);
                }
                if (k + 1 < 2 * n) pages.load(p.at, w.e, (w.t0 + Order::use(k + 1, n).i) * kT, tokens);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(m.full + ring.i))
                         : "memory");
            ring.next();
        }
        if (!ok) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Loader warps of 8-bit caches (256 threads): codes come into registers DEPTH
// tiles ahead, are widened there and stored to their stage (a copy to shared
// memory first would cost the tile two more passes through it, which is what
// bounds 8-bit tiles).
template <int D, int NS, int QR, typename Order, int DEPTH>
__device__ __forceinline__ void load_e4m3(const TreeParams& p, const TcRing& m, const Waiter& wait, TreeCursor cur,
                                          long long u, long long end, int tid) {
    constexpr int kC8 = D / 16, kMine = kT * kC8 / 256, kStep = 256 / kC8;  // 16-code chunks of a row, of a thread
    const int c = tid % kC8, r0 = tid / kC8;
    Ring<NS> ring;
    uint32_t q_ph = 1;
    // reads run over the same pieces and tiles, ahead of the widening
    TreeCursor acur = cur;
    long long au = u;
    TreePiece aw, w;
    int a_n = 0, a_k = 0, n = 0, k = 0;  // tiles of the piece, place in their order
    bool a_more = true;
    TilePages pages;  // of the next tile to read
    auto advance = [&](TreeCursor& cc, long long& uu, TreePiece& ww, int& nn, int& kk) {
        while (kk >= 2 * nn) {  // the next piece with rows
            if (!next_piece(p, cc, uu, end, ww)) return false;
            if (ww.nodes * p.G - ww.mt * p.tile_rows > 0) { nn = ww.t1 - ww.t0; kk = 0; }
        }
        return true;
    };
    auto read = [&](uint4 (&x)[kMine]) {
        if (!a_more) return;
        const int before = a_k;
        a_more = advance(acur, au, aw, a_n, a_k);
        if (!a_more) return;
        const int tokens = aw.prefix + aw.nodes;
        if (p.at.block_table && (before != a_k || a_k == 0)) pages.load(p.at, aw.e, aw.t0 * kT, tokens);
        const RingUse use = Order::use(a_k++, a_n);
        const int tok0 = (aw.t0 + use.i) * kT;
        const uint8_t* src = static_cast<const uint8_t*>(use.is_v ? p.v : p.k) + c * 16;
#pragma unroll
        for (int y = 0; y < kMine; ++y) {
            const int r = r0 + y * kStep, t = min(tok0 + r, tokens - 1);
            const long long row = p.at.block_table ? pages.row(p.at, aw.e, aw.h, t, r)
                                                   : ((long long)aw.e * p.at.hkv + aw.h) * p.at.s_cap + t;
            x[y] = tok0 + r < tokens ? ldg_stream16(src + row * D) : make_uint4(0, 0, 0, 0);
        }
        if (p.at.block_table && a_k < 2 * a_n) pages.load(p.at, aw.e, (aw.t0 + Order::use(a_k, a_n).i) * kT, tokens);
    };
    auto step = [&](uint4 (&x)[kMine]) {  // widens and stores one tile, reads a later one in its place
        const int before = k;
        if (!advance(cur, u, w, n, k)) return false;
        if (before != k || k == 0) {
            if (!__all_sync(0xffffffffu, wait(m.q_empty, q_ph))) return false;
            q_ph ^= 1;
            load_queries<D, QR, 256>(p, w, m.q, tid, false);
        }
        ++k;
        if (!__all_sync(0xffffffffu, wait(m.empty + ring.i, ring.ph ^ 1))) return false;
        uint8_t* dst = m.stages + ring.i * (kT * D * 2);
#pragma unroll
        for (int y = 0; y < kMine; ++y) {
            const int r = r0 + y * kStep;
            const uint2 a = widen4(x[y].x), b = widen4(x[y].y), d = widen4(x[y].z), f = widen4(x[y].w);
            *reinterpret_cast<uint4*>(dst + tile_at(r, 2 * c)) = make_uint4(a.x, a.y, b.x, b.y);
            *reinterpret_cast<uint4*>(dst + tile_at(r, 2 * c + 1)) = make_uint4(d.x, d.y, f.x, f.y);
        }
        proxy_fence();
        mbar_arrive(m.full + ring.i);
        ring.next();
        read(x);
        return true;
    };
    uint4 x[DEPTH][kMine];
#pragma unroll
    for (int y = 0; y < DEPTH; ++y) read(x[y]);
    for (bool ok = true; ok;) {
#pragma unroll
        for (int y = 0; y < DEPTH; ++y) {
            ok = step(x[y]);
            if (!ok) break;
        }
    }
}

}  // namespace

}  // namespace ds
