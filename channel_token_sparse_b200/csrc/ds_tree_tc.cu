// ds_tree_tc.cu -- tree attention over bf16 and 8-bit caches on the tensor
// cores (tcgen05, accumulators in tensor memory), for sm_100a.
//
// One persistent CTA per SM walks its share of units (ds_tree.cuh). For a tile
// of 128 tokens and 128 query rows: S = Q K^T into tensor memory, weights
// P = 2^(qscale S - m) in bf16 back into tensor memory (over S), O += P V. The
// running maximum m moves only when a tile's maximum passes it by 8 (a factor
// 2^8, far inside fp32 and bf16), so O is rarely rescaled.
//
// Two streams of tiles are in flight, each with its own S, O and softmax
// warpgroup: while one's weights are formed the other's products run. Up to
// 128 query rows (MT = 1): the streams take alternate token tiles of the same
// rows and are joined at the end; more rows (MT = 2): each stream has 128 rows
// and both use every token tile, which halves the reads a row costs.
//
// Roles: warps 0-3 and 4-7 softmax of stream 0 and 1 (a thread a row), warp 8
// issues the products, warps 12 on bring K and V tiles into a ring of
// 128-byte-swizzled stages by 16-byte asynchronous copies (any page size;
// rows past the sequence become zeros). 8-bit tiles are copied as they are
// into the loaders' own slots, widened to bf16 (exact) and stored into the
// ring; the rows' scales multiply S and P.
//
// The products take every row of V with every weight, and 0 * NaN is NaN, so
// the rows of tree nodes (which some query rows may not see) are looked
// through for values that are not finite; such values are zeroed in the stage
// and added to the rows that do see them at the end. An 8-bit tree row whose
// scales are not finite is set aside the same way.
#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kT = 128;  // tokens of a tile, and rows of a row block

template <int TYPE, int D, int MT>
struct Cfg {
    static constexpr bool kQ8 = TYPE == kTreeE4M3;
    static constexpr int kLoadWarps = kQ8 ? 8 : 4;
    static constexpr int kThreads = (12 + kLoadWarps) * 32;
    // Registers of a thread by role: 512 (8-bit: 640) threads are launched with
    // 128 (96) each, and the four-warp groups redistribute them: their sums are
    // 168 + 168 + 72 + 104 = 4 * 128 and 136 + 136 + 64 + 2 * 72 = 5 * 96.
    static constexpr int kRegSoftmax = kQ8 ? 136 : 168, kRegMma = kQ8 ? 64 : 72, kRegLoad = kQ8 ? 72 : 104;
    static_assert(2 * kRegSoftmax + kRegMma + (kQ8 ? 2 : 1) * kRegLoad <= (kQ8 ? 5 * 96 : 4 * 128), "registers");
    static constexpr int kStage = kT * D * 2;       // bytes of a K or V tile in bf16
    static constexpr int kQ = MT * kT * D * 2;
    static constexpr int kRaw = kQ8 ? (D == 128 ? 3 : 6) : 0;
    static constexpr int kRawBytes = kT * D;
    static constexpr int kScale = kQ8 ? 8 * 2 * kT * 4 : 0;  // a softmax warp's K and V scales of a tile
    static constexpr int kStages = D == 128 ? (kQ8 ? 5 : 7) - MT : (kQ8 ? 9 : 13) - MT;
    static constexpr int oStage = kQ, oRaw = oStage + kStages * kStage, oScale = oRaw + kRaw * kRawBytes;
    static constexpr int oMl = oScale + kScale;             // [2][128] maxima, [2][128] sums
    static constexpr int oBar = oMl + 4 * kT * 4;
    static constexpr int kBars = 2 * kStages + 9;
    static constexpr int kSmem = oBar + kBars * 8 + 64;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

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

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
          "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
          "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets (in 16-byte units), version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)(addr >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: bf16 x bf16 -> f32, M = 128, B of N columns, K-major
// or (transposed) N-major.
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool b_n_major) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_n_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
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
// of 64 channels, rows of 128 bytes, chunks exchanged within groups of 8 rows.
__device__ __forceinline__ int tile_at(int r, int c) { return (c >> 3) * (kT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

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

// The order in which a piece of n token tiles uses the ring: the k-th of its
// 2n uses is token tile `i`, of V or K. MT = 1: K0 K1, then V_i K_{i+2};
// MT = 2: K_i V_i.
struct RingUse { int i; bool is_v; };
template <int MT> __device__ __forceinline__ RingUse ring_use(int k, int n) {
    if (MT == 2) return RingUse{k >> 1, (k & 1) != 0};
    const int lead = n > 1 ? 2 : 1, j = k - lead;
    if (j < 0) return RingUse{k, false};
    if (j < 2 * (n - 2)) return RingUse{(j & 1) ? 2 + j / 2 : j / 2, (j & 1) == 0};
    return RingUse{k - n, true};  // the last V tiles
}
// The use of the ring that holds V of token tile i.
template <int MT> __device__ __forceinline__ int v_use(int i, int n) {
    return MT == 2 ? 2 * i + 1 : n == 1 ? 1 : i < n - 1 ? 2 * i + 2 : 2 * i + 1;
}

// -------------------------------------------------------------------- kernel

template <int TYPE, int D, int MT>
__global__ void __launch_bounds__(Cfg<TYPE, D, MT>::kThreads, 1) ds_tree_tc_kernel(const __grid_constant__ TreeParams p) {
    using C = Cfg<TYPE, D, MT>;
    constexpr int NS = C::kStages;
    constexpr int kChunks = D / 8;  // 16-byte chunks of a bf16 row
    extern __shared__ __align__(1024) uint8_t smem[];
    float* ml = reinterpret_cast<float*>(smem + C::oMl);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::oBar);
    uint64_t* empty = full + NS;
    uint64_t* s_full = empty + NS;   // [2] S of a stream is there
    uint64_t* p_full = s_full + 2;   // [2] its P is, and O is ready to take it
    uint64_t* o_done = p_full + 2;   // [2] O has taken it
    uint64_t* q_empty = o_done + 2;  // the piece's S products are done
    uint64_t* xch = q_empty + 1;     // softmax warps among themselves
    uint64_t* drain = xch + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* bad = tmem_slot + 2;   // [8] nodes whose V row holds values that are not finite

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, C::kLoadWarps * 32);
            mbar_init(empty + i, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full + s, 1);
            mbar_init(p_full + s, 128);
            mbar_init(o_done + s, 1);
        }
        mbar_init(q_empty, 1);
        mbar_init(xch, 256);
        mbar_init(drain, 1);
        *stop = 0;
        for (int i = 0; i < 8; ++i) bad[i] = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Waiter wait{stop, p.err};

    const TreeShares shares(tree_total(p), p.grid);
    long long u = shares.begin(blockIdx.x);
    const long long end = shares.begin(blockIdx.x + 1);
    TreeCursor cur;
    if (u < end) cur = tree_seek(p, u);
    TreePiece w;

    if (warp >= 12) {
        // ------------------------------------------------------------ loaders
        reg_dec<C::kRegLoad>();
        const int tid = threadIdx.x - 12 * 32;
        Ring<NS> ring;
        uint32_t q_ph = 1;  // the first wait on q_empty passes
        if constexpr (!C::kQ8) {
            const int c = tid % kChunks, r0 = tid / kChunks;
            constexpr int kStep = 128 / kChunks;  // rows the 128 threads cover at a time
            while (next_piece(p, cur, u, end, w)) {
                const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
                if (rows <= 0) continue;
                const int n = w.t1 - w.t0, tokens = w.prefix + w.nodes;
                // the queries come with the first K tile
                if (!__all_sync(0xffffffffu, wait(q_empty, q_ph))) break;
                q_ph ^= 1;
#pragma unroll 4
                for (int k = 0; k < MT * kChunks; ++k) {
                    const int row = r0 + k * kStep;
                    const bool there = row < rows;
                    const size_t at = there ? q_offset(p, w.e, w.h, row0 + row, D) : 0;
                    cp_async16_zfill(smem + (row / kT) * kT * D * 2 + tile_at(row % kT, c),
                                     static_cast<const uint16_t*>(p.q) + at + c * 8, there);
                }
                bool ok = true;
                TilePages pages;
                if (p.at.block_table) pages.load(p.at, w.e, w.t0 * kT, tokens);
                for (int k = 0; k < 2 * n; ++k) {
                    const RingUse use = ring_use<MT>(k, n);
                    ok = __all_sync(0xffffffffu, wait(empty + ring.i, ring.ph ^ 1));
                    if (!ok) break;
                    const uint32_t dst = smem_u32(smem + C::oStage + ring.i * C::kStage);
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
                        if (k + 1 < 2 * n) pages.load(p.at, w.e, (w.t0 + ring_use<MT>(k + 1, n).i) * kT, tokens);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + ring.i))
                                 : "memory");
                    ring.next();
                }
                if (!ok) break;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            // Each thread widens the codes that it copied itself: four 16-code
            // chunks of a tile (two for 64 channels), kRaw - 1 tiles ahead.
            constexpr int kC8 = D / 16, kMine = kT * kC8 / 256, kStep = 256 / kC8;
            const int c = tid % kC8, r0 = tid / kC8;
            uint8_t* raw = smem + C::oRaw + tid * 16;
            // copies run over the same pieces and tiles, ahead of the widening
            TreeCursor acur = cur;
            long long au = u;
            TreePiece aw;
            int a_n = 0, a_k = 0, a_slot = 0;  // tiles of its piece, place in their order, slot
            bool a_more = true;
            TilePages pages;  // of the next tile to copy
            auto issue = [&] {
                while (a_more && a_k >= 2 * a_n) {  // the next piece with rows
                    a_more = next_piece(p, acur, au, end, aw);
                    if (a_more && aw.nodes * p.G - aw.mt * p.tile_rows > 0) {
                        a_n = aw.t1 - aw.t0;
                        a_k = 0;
                        if (p.at.block_table) pages.load(p.at, aw.e, aw.t0 * kT, aw.prefix + aw.nodes);
                    }
                }
                if (a_more) {
                    const RingUse use = ring_use<MT>(a_k++, a_n);
                    const int tok0 = (aw.t0 + use.i) * kT, tokens = aw.prefix + aw.nodes;
                    const uint8_t* src = static_cast<const uint8_t*>(use.is_v ? p.v : p.k) + c * 16;
                    const uint32_t dst = smem_u32(raw + a_slot * C::kRawBytes);
#pragma unroll
                    for (int x = 0; x < kMine; ++x) {
                        const int r = r0 + x * kStep, t = min(tok0 + r, tokens - 1);
                        const long long row = p.at.block_table ? pages.row(p.at, aw.e, aw.h, t, r)
                                                               : ((long long)aw.e * p.at.hkv + aw.h) * p.at.s_cap + t;
                        copy16(dst + x * 4096, src + row * D, tok0 + r < tokens);
                    }
                    if (p.at.block_table && a_k < 2 * a_n)
                        pages.load(p.at, aw.e, (aw.t0 + ring_use<MT>(a_k, a_n).i) * kT, tokens);
                }
                cp_async_commit();
                if (++a_slot == C::kRaw) a_slot = 0;
            };
            for (int k = 0; k < C::kRaw - 1; ++k) issue();
            int slot = 0;
            while (next_piece(p, cur, u, end, w)) {
                const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
                if (rows <= 0) continue;
                const int n = w.t1 - w.t0;
                if (!__all_sync(0xffffffffu, wait(q_empty, q_ph))) break;
                q_ph ^= 1;
                const int qc = tid % kChunks, qr = tid / kChunks;
#pragma unroll 4
                for (int k = 0; k < MT * kT * kChunks / 256; ++k) {
                    const int row = qr + k * (256 / kChunks);
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row < rows)
                        x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                            q_offset(p, w.e, w.h, row0 + row, D) + qc * 8);
                    *reinterpret_cast<uint4*>(smem + (row / kT) * kT * D * 2 + tile_at(row % kT, qc)) = x;
                }
                bool ok = true;
                for (int k = 0; k < 2 * n; ++k) {
                    issue();
                    ok = __all_sync(0xffffffffu, wait(empty + ring.i, ring.ph ^ 1));
                    if (!ok) break;
                    cp_async_wait<C::kRaw - 1>();
                    uint8_t* dst = smem + C::oStage + ring.i * C::kStage;
#pragma unroll
                    for (int x = 0; x < kMine; ++x) {
                        const int r = r0 + x * kStep;
                        const uint4 y = *reinterpret_cast<const uint4*>(raw + slot * C::kRawBytes + x * 4096);
                        const uint2 a = widen4(y.x), b = widen4(y.y), d = widen4(y.z), f = widen4(y.w);
                        *reinterpret_cast<uint4*>(dst + tile_at(r, 2 * c)) = make_uint4(a.x, a.y, b.x, b.y);
                        *reinterpret_cast<uint4*>(dst + tile_at(r, 2 * c + 1)) = make_uint4(d.x, d.y, f.x, f.y);
                    }
                    proxy_fence();
                    mbar_arrive(full + ring.i);
                    ring.next();
                    if (++slot == C::kRaw) slot = 0;
                }
                if (!ok) break;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp >= 8) {
        // ----------------------------------------------------------- products
        reg_dec<C::kRegMma>();
        if (warp > 8) u = end;  // one warp issues; its group's others only gave registers back
        Ring<NS> ring;
        uint32_t p_ph[2] = {0, 0};
        constexpr uint32_t kS = instr_desc(kT, false), kO = instr_desc(D, true);
        const uint32_t q_addr = smem_u32(smem), st_addr = smem_u32(smem + C::oStage);
        auto s_of = [&](int s) { return tmem + s * kT; };
        auto o_of = [&](int s) { return tmem + 2 * kT + s * D; };
        // The whole warp walks along, so addresses stay warp-uniform; one lane issues.
        auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        auto ready = [&](const Ring<NS>& r) {
            if (!all_wait(full + r.i, r.ph)) return false;
            proxy_fence();  // the copies' writes, before the products read them
            return true;
        };
        auto commit = [&](uint64_t* bar) { if (elected()) tc_commit(bar); };
        auto scores = [&](int s, int stage) {  // S = Q K^T of stream s
            const uint32_t d = s_of(s);
            const uint64_t a = smem_desc(q_addr + (MT == 2 ? s : 0) * kT * D * 2, 16, 1024);
            const uint64_t b = smem_desc(st_addr + stage * C::kStage, 16, 1024);
            if (elected()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (kT * 128) + (k & 3) * 32) >> 4;
                    mma_ss(d, a + off, b + off, kS, k > 0);
                }
                tc_commit(s_full + s);
            }
        };
        auto values = [&](int s, int stage, bool add) {  // O += P V of stream s
            const uint32_t d = o_of(s), a = s_of(s);
            const uint64_t b = smem_desc(st_addr + stage * C::kStage, kT * 128, 1024);
            if (elected()) {
#pragma unroll
                for (int k = 0; k < kT / 16; ++k) mma_ts(d, a + k * 8, b + k * 128, kO, add || k > 0);
                tc_commit(o_done + s);
            }
        };
        auto weights = [&](int s) {  // P of stream s is there
            if (!all_wait(p_full + s, p_ph[s])) return false;
            p_ph[s] ^= 1;
            tc_fence_after();
            return true;
        };
        while (next_piece(p, cur, u, end, w)) {
            if (w.nodes * p.G - w.mt * p.tile_rows <= 0) continue;
            const int n = w.t1 - w.t0;
            bool ok = true;
            if (MT == 1) {
                // S of the first two tiles, then PV of tile i and S of tile i + 2
                for (int i = -2; ok && i < n; ++i) {
                    if (i >= 0) {
                        ok = ready(ring) && weights(i & 1);
                        if (!ok) break;
                        values(i & 1, ring.i, i >= 2);
                        commit(empty + ring.i);
                        ring.next();
                    }
                    if (i + 2 < n) {
                        ok = ready(ring);
                        if (!ok) break;
                        scores(i & 1, ring.i);
                        commit(empty + ring.i);
                        if (i + 3 == n) commit(q_empty);
                        ring.next();
                    }
                }
            } else {
                // of each stream: PV of tile i, then S of tile i + 1
                Ring<NS> rv = ring;
                for (int i = -1; ok && i < n; ++i) {
                    const bool more = i + 1 < n;
                    if (i >= 0) { rv = ring; ring.next(); }
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (i >= 0) {
                            ok = (s > 0 || ready(rv)) && weights(s);
                            if (!ok) break;
                            values(s, rv.i, i > 0);
                        }
                        if (more) {
                            ok = s > 0 || ready(ring);
                            if (!ok) break;
                            scores(s, ring.i);
                        }
                    }
                    if (!ok) break;
                    if (i >= 0) commit(empty + rv.i);
                    if (more) {
                        commit(empty + ring.i);
                        if (i + 2 == n) commit(q_empty);
                        ring.next();
                    }
                }
            }
            if (!ok) {  // products in flight end before the tensor memory is given back
                commit(drain);
                mbar_wait_bounded(drain, 0, p.err, 3, 10000000ull);
                break;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        reg_inc<C::kRegSoftmax>();
        // a wait that all lanes leave with the same answer
        auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        const int st = warp >> 2;                   // stream
        const int r = (warp & 3) * 32 + lane;       // row of the row block
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + st * kT, t_o = tmem + lanes + 2 * kT;
        float* ks = reinterpret_cast<float*>(smem + C::oScale) + warp * 2 * kT;
        float* vs = ks + kT;
        uint32_t s_ph = 0, o_cnt = 0, x_ph = 0;     // o_cnt: products awaited or due on o_done
        Ring<NS> vring;                             // the V stages, for the looks at tree rows
        long long uses = 0;                         // ring uses of the pieces before
        bool ok = true;
        while (ok && next_piece(p, cur, u, end, w)) {
            const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
            if (rows <= 0) continue;
            const int n = w.t1 - w.t0, tokens = w.prefix + w.nodes;
            const int item_row = (MT == 2 ? st * kT : 0) + r;
            const bool live = item_row < rows;
            const bool warp_live = (item_row - lane) < rows;
            const int node = (row0 + item_row) / p.G;
            float m = -INFINITY, l = 0.f;
            int done = 0;  // tiles of this stream
            constexpr int kEvery = MT == 1 ? 2 : 1;  // token tiles from one of this stream's to its next
            const int i0 = MT == 1 ? st : 0;
            // scales of a tile's rows (8-bit): lane l has rows l, l + 32 ..; 0 past the sequence
            float sc_k[kT / 32], sc_v[kT / 32];
            auto scales = [&](int tok) {
#pragma unroll
                for (int k = 0; k < kT / 32; ++k) {
                    const int t = tok + k * 32 + lane;
                    const bool there = t < tokens;
                    const long long row = there ? tree_row(p.at, w.e, w.h, t) : 0;
                    sc_k[k] = there ? __ldg(p.k_scale + row) : 0.f;
                    sc_v[k] = there ? __ldg(p.v_scale + row) : 0.f;
                }
            };
            if (C::kQ8 && i0 < n) scales((w.t0 + i0) * kT);
            for (int i = i0; i < n; i += kEvery) {
                const int tok0 = (w.t0 + i) * kT;
                const bool masked = tok0 + kT > w.prefix;
                if constexpr (C::kQ8) {  // the tile's scales; those of the stream's next tile are read meanwhile
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kT / 32; ++k) {
                        const int j = tok0 + k * 32 + lane - w.prefix;
                        float a = sc_k[k] * p.qscale, b = sc_v[k];
                        if (j >= 0 && !(isfinite(a) && isfinite(b))) {  // a tree row, not seen by all: set aside
                            a = b = 0.f;
                            atomicOr(bad + (j >> 5), 1u << (j & 31));
                        }
                        ks[k * 32 + lane] = a;
                        vs[k * 32 + lane] = b;
                    }
                    __syncwarp();
                    if (i + kEvery < n) scales(tok0 + kEvery * kT);
                }
                if (masked) {
                    // values of tree rows that are not finite leave the stage (see the top)
                    const long long use = uses + v_use<MT>(i, n);
                    const int stage = (int)(use % NS);
                    ok = all_wait(full + stage, (uint32_t)(use / NS) & 1);
                    if (!ok) break;
                    uint8_t* v = smem + C::oStage + stage * C::kStage;
                    const int b = max(w.prefix - tok0, 0), cnt = min(tokens - tok0, kT) - b;
                    bool patched = false;
                    for (int x = (warp & 3) * 32 + lane; x < cnt * kChunks; x += 128) {
                        const int vr = b + x / kChunks;
                        uint32_t* at = reinterpret_cast<uint32_t*>(v + tile_at(vr, x % kChunks));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t y = at[k];
                            const bool lo = (y & 0x7f80u) == 0x7f80u, hi = (y & 0x7f800000u) == 0x7f800000u;
                            if (lo || hi) {
                                at[k] = y & (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
                                const int j = tok0 + vr - w.prefix;
                                atomicOr(bad + (j >> 5), 1u << (j & 31));
                                patched = true;
                            }
                        }
                    }
                    if (patched) proxy_fence();
                }
                ok = all_wait(s_full + st, s_ph);
                if (!ok) break;
                s_ph ^= 1;
                tc_fence_after();
                if (warp_live) {
                    if (masked) {  // what a row does not see gets the score -infinity
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t vis = live ? visible(p, w.e, node, w.nodes, tok0 + 32 * k - w.prefix) : 0u;
                            uint32_t x[32];
                            tc_ld32(x, t_s + 32 * k);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                float f = __uint_as_float(x[j]);
                                if constexpr (C::kQ8) f *= ks[32 * k + j];
                                x[j] = (vis >> j & 1) ? __float_as_uint(f) : 0xff800000u;
                            }
                            tc_st32(t_s + 32 * k, x);
                        }
                        tc_wait_st();
                        if constexpr (C::kQ8) {  // the scales are in these scores
                            __syncwarp();
                            for (int k = lane; k < kT; k += 32) ks[k] = 1.f;
                            __syncwarp();
                        }
                    }
                    // the tile's maximum
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int k = 0; k < 4; k += 2) {
                        uint32_t x[2][32];
                        tc_ld32(x[0], t_s + 32 * k);
                        tc_ld32(x[1], t_s + 32 * k + 32);
                        tc_wait_ld();
                        float a[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int j = 0; j < 64; j += 4) {
                            float f[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) f[q] = __uint_as_float(x[j >> 5][(j & 31) + q]);
                            if constexpr (C::kQ8) {
                                const float4 sc = *reinterpret_cast<const float4*>(ks + 32 * k + j);
                                f[0] *= sc.x; f[1] *= sc.y; f[2] *= sc.z; f[3] *= sc.w;
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) a[q] = fmaxf(a[q], f[q]);
                        }
                        mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                    }
                    if constexpr (!C::kQ8) mx *= p.qscale;
                    if (done == 0) {
                        m = mx;
                    } else {
                        const bool move = mx > m + 8.f;
                        if (__any_sync(0xffffffffu, move)) {
                            // the products of this stream before are done; nothing else touches O
                            ok = all_wait(o_done + st, (o_cnt - 1) & 1);
                            if (!ok) break;
                            tc_fence_after();
                            const float f = move ? (m == -INFINITY ? 0.f : ex2(m - mx)) : 1.f;
                            if (move) m = mx;
                            l *= f;
#pragma unroll
                            for (int k = 0; k < D / 32; ++k) {
                                uint32_t x[32];
                                tc_ld32(x, t_o + st * D + 32 * k);
                                tc_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                                tc_st32(t_o + st * D + 32 * k, x);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : -m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int k = 0; k < 4; k += 2) {
                        uint32_t x[2][32];
                        tc_ld32(x[0], t_s + 32 * k);
                        tc_ld32(x[1], t_s + 32 * k + 32);
                        tc_wait_ld();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t y[16];
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                float f[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q) f[q] = __uint_as_float(x[h][j + q]);
                                if constexpr (C::kQ8) {
                                    const float4 sc = *reinterpret_cast<const float4*>(ks + 32 * (k + h) + j);
                                    f[0] = fmaf(f[0], sc.x, base); f[1] = fmaf(f[1], sc.y, base);
                                    f[2] = fmaf(f[2], sc.z, base); f[3] = fmaf(f[3], sc.w, base);
                                } else {
#pragma unroll
                                    for (int q = 0; q < 4; ++q) f[q] = fmaf(f[q], p.qscale, base);
                                }
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    f[q] = ex2(f[q]);
                                    sum[q] += f[q];
                                }
                                if constexpr (C::kQ8) {
                                    const float4 sc = *reinterpret_cast<const float4*>(vs + 32 * (k + h) + j);
                                    f[0] *= sc.x; f[1] *= sc.y; f[2] *= sc.z; f[3] *= sc.w;
                                }
                                y[j / 2] = pack_bf16x2(f[0], f[1]);
                                y[j / 2 + 1] = pack_bf16x2(f[2], f[3]);
                            }
                            tc_st16(t_s + 16 * (k + h), y);
                        }
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc_wait_st();
                }
                tc_fence_before();
                mbar_arrive(p_full + st);
                ++o_cnt;
                ++done;
            }
            if (!ok) break;
            uses += 2 * n;
            // the piece's result
            if (done > 0) {
                ok = all_wait(o_done + st, (o_cnt - 1) & 1);
                if (!ok) break;
            }
            ml[st * kT + r] = m;
            ml[(2 + st) * kT + r] = l;
            tc_fence_before();
            mbar_arrive(xch);
            ok = all_wait(xch, x_ph);
            if (!ok) break;
            x_ph ^= 1;
            tc_fence_after();
            uint32_t any_bad = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) any_bad |= bad[k];
            if (warp_live) {
                // MT = 1: both streams' rows are joined, and each warpgroup takes half of the channels
                float f0 = 1.f, f1 = 0.f, mm = m, ll = l;
                if (MT == 1) {
                    const float m0 = ml[r], m1 = n > 1 ? ml[kT + r] : -INFINITY;
                    mm = fmaxf(m0, m1);
                    const float base = mm == -INFINITY ? 0.f : mm;
                    f0 = ex2(m0 - base);
                    f1 = n > 1 ? ex2(m1 - base) : 0.f;
                    ll = ml[2 * kT + r] * f0 + (n > 1 ? ml[3 * kT + r] * f1 : 0.f);
                }
                const bool whole = w.whole();
                const float inv = whole ? (ll == 0.f ? 0.f : 1.f / ll) : 1.f;
                float* part = part_of(p, blockIdx.x, w.t0 == 0, D);
                const size_t at = live ? q_offset(p, w.e, w.h, row0 + item_row, D) : 0;
                constexpr int kCols = MT == 1 ? D / 2 : D;
                const int col0 = MT == 1 ? st * kCols : 0;
                if (live && !whole && (MT == 2 || st == 0)) {
                    part[item_row] = mm;
                    part[p.part_rows + item_row] = ll;
                }
#pragma unroll 1
                for (int k = 0; k < kCols / 32; ++k) {
                    const int col = col0 + 32 * k;
                    uint32_t x[32];
                    float o[32];
                    tc_ld32(x, t_o + (MT == 2 ? st * D : 0) + col);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(x[j]) * f0;
                    if (MT == 1 && n > 1) {
                        tc_ld32(x, t_o + D + col);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(x[j]), f1, o[j]);
                    }
                    if (!live) continue;
                    if (any_bad) {
                        for (int q = 0; q < 8; ++q) {
                            if (!bad[q]) continue;
                            uint32_t see = bad[q] & mask_word(p, w.e, node, q);
                            for (; see; see &= see - 1) {
                                const long long row = tree_row(p.at, w.e, w.h, w.prefix + 32 * q + __ffs(see) - 1);
                                bool fine = true;
                                if constexpr (C::kQ8)
                                    fine = isfinite(p.k_scale[row] * p.qscale) && isfinite(p.v_scale[row]);
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    float f;
                                    if constexpr (C::kQ8) {  // NaN in a channel, or throughout by its row's scales
                                        const uint8_t code = static_cast<const uint8_t*>(p.v)[row * D + col + j];
                                        f = (code & 0x7f) == 0x7f || !fine ? NAN : 0.f;
                                    } else {
                                        f = Elem<bf16_t>::to_f32(static_cast<const bf16_t*>(p.v)[row * D + col + j]);
                                        f = isfinite(f) ? 0.f : f;
                                    }
                                    o[j] += f;
                                }
                            }
                        }
                    }
                    if (!whole) {
                        float4* d = reinterpret_cast<float4*>(part + 2 * p.part_rows + (size_t)item_row * D + col);
#pragma unroll
                        for (int j = 0; j < 8; ++j) d[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    } else if (p.out_bf16) {
                        uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at + col);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            d[j] = make_uint4(pack_bf16x2(o[8 * j] * inv, o[8 * j + 1] * inv),
                                              pack_bf16x2(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                              pack_bf16x2(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                                              pack_bf16x2(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
                    } else {
                        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at + col);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            d[j] = make_float4(o[4 * j] * inv, o[4 * j + 1] * inv, o[4 * j + 2] * inv, o[4 * j + 3] * inv);
                    }
                }
            }
            // both streams have read O, the maxima and the marks before either goes on
            tc_fence_before();
            mbar_arrive(xch);
            ok = all_wait(xch, x_ph);
            if (!ok) break;
            x_ph ^= 1;
            if (any_bad && threadIdx.x < 8) bad[threadIdx.x] = 0;
            if (any_bad) {  // cleared before the next piece marks
                mbar_arrive(xch);
                ok = all_wait(xch, x_ph);
                x_ph ^= 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int TYPE, int D, int MT>
cudaError_t run(const TreeParams& p, cudaStream_t st) {
    using C = Cfg<TYPE, D, MT>;
    cudaError_t e = cudaFuncSetAttribute(ds_tree_tc_kernel<TYPE, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
    ds_tree_tc_kernel<TYPE, D, MT><<<p.grid, C::kThreads, C::kSmem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

TreePlan plan_tree_tc(int rows, int d) {
    (void)d;
    return TreePlan{rows <= kT ? kT : 2 * kT, kT, 148};
}

cudaError_t launch_tree_tc(const TreeParams& p, int type, int d, cudaStream_t st) {
    const bool two = p.tile_rows == 2 * kT;
#define DS_T(TY, D_) (two ? run<TY, D_, 2>(p, st) : run<TY, D_, 1>(p, st))
    if (type == kTreeBF16) return d == 64 ? DS_T(kTreeBF16, 64) : DS_T(kTreeBF16, 128);
    return d == 64 ? DS_T(kTreeE4M3, 64) : DS_T(kTreeE4M3, 128);
#undef DS_T
}

}  // namespace ds
