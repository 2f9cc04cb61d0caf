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
// issues the products, the others bring K and V tiles into a ring of
// 128-byte-swizzled stages by 16-byte asynchronous copies (any page size;
// rows past the sequence become zeros). 8-bit tiles are copied as they are
// into the loaders' own slots, widened to bf16 (exact) and stored into the
// ring; the rows' scales multiply S and P.
//
// The products take every row of V with every weight, and 0 * NaN is NaN, so
// the rows of tree nodes (which some query rows may not see) are looked
// through for values that are not finite; such values are zeroed in the stage
// and added to the rows that do see them at the end.
#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kT = 128;  // tokens of a tile, and rows of a row block

template <int TYPE, int D, int MT>
struct Cfg {
    static constexpr bool kQ8 = TYPE == kTreeE4M3;
    static constexpr int kLoadWarps = kQ8 ? 8 : 4;
    static constexpr int kThreads = (9 + kLoadWarps) * 32;
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
        if (mbar_try_wait(bar, parity)) return true;
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

// Four e4m3 codes -> four bf16 values (exact).
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y));
}

// The order in which a piece of n token tiles uses the ring. MT = 1: K0 K1,
// then V_i K_{i+2}; MT = 2: K_i V_i. Calls f(token tile, is V).
template <int MT, typename F>
__device__ __forceinline__ bool ring_order(int n, F f) {
    if (MT == 1) {
        if (!f(0, false)) return false;
        if (n > 1 && !f(1, false)) return false;
        for (int i = 0; i < n; ++i) {
            if (!f(i, true)) return false;
            if (i + 2 < n && !f(i + 2, false)) return false;
        }
    } else {
        for (int i = 0; i < n; ++i)
            if (!f(i, false) || !f(i, true)) return false;
    }
    return true;
}

// -------------------------------------------------------------------- kernel

template <int TYPE, int D, int MT>
__global__ void __launch_bounds__(Cfg<TYPE, D, MT>::kThreads, 1) ds_tree_tc_kernel(const TreeParams p) {
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

    const long long total = tree_total(p);
    long long u = share_begin(total, blockIdx.x, p.grid);
    const long long end = share_begin(total, blockIdx.x + 1, p.grid);
    TreeCursor cur;
    if (u < end) cur = tree_seek(p, u);
    TreePiece w;

    if (warp >= 9) {
        // ------------------------------------------------------------ loaders
        const int tid = threadIdx.x - 9 * 32;
        Ring<NS> ring;
        uint32_t q_ph = 1;  // the first wait on q_empty passes
        if constexpr (!C::kQ8) {
            const int c = tid % kChunks, r0 = tid / kChunks;
            constexpr int kStep = 128 / kChunks;  // rows the 128 threads cover at a time
            bool ok = true;
            while (ok && next_piece(p, cur, u, end, w)) {
                const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
                if (rows <= 0) continue;
                const int tokens = w.prefix + w.nodes;
                bool first = true;
                ok = ring_order<MT>(w.t1 - w.t0, [&](int i, bool is_v) {
                    if (first) {  // the queries go with the first K tile
                        first = false;
                        if (!wait(q_empty, q_ph)) return false;
                        q_ph ^= 1;
                        for (int b = 0; b < MT; ++b)
#pragma unroll 4
                            for (int k = 0; k < kChunks; ++k) {
                                const int r = r0 + k * kStep, row = b * kT + r;
                                const bool there = row < rows;
                                const size_t at = there ? q_offset(p, w.e, w.h, row0 + row, D) : 0;
                                cp_async16_zfill(smem + b * kT * D * 2 + tile_at(r, c),
                                                 static_cast<const uint16_t*>(p.q) + at + c * 8, there);
                            }
                    }
                    if (!wait(empty + ring.i, ring.ph ^ 1)) return false;
                    uint8_t* dst = smem + C::oStage + ring.i * C::kStage;
                    const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.v : p.k) + c * 8;
                    const int tok0 = (w.t0 + i) * kT;
#pragma unroll
                    for (int k = 0; k < kChunks; ++k) {
                        const int r = r0 + k * kStep;
                        const bool there = tok0 + r < tokens;
                        const long long row = there ? tree_row(p.at, w.e, w.h, tok0 + r) : 0;
                        cp_async16_zfill(dst + tile_at(r, c), src + row * D, there);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + ring.i))
                                 : "memory");
                    ring.next();
                    return true;
                });
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
            auto a_next = [&](int& i, bool& is_v) {  // the next tile in ring order
                for (;;) {
                    if (a_k < 2 * a_n) break;
                    if (!a_more || !next_piece(p, acur, au, end, aw)) { a_more = false; return false; }
                    if (aw.nodes * p.G - aw.mt * p.tile_rows <= 0) continue;
                    a_n = aw.t1 - aw.t0;
                    a_k = 0;
                }
                const int k = a_k++;
                if (MT == 2) { i = k >> 1; is_v = k & 1; return true; }
                // K0 K1 V0 K2 V1 K3 ... V_{n-2} V_{n-1}; one tile: K0 V0
                if (k < 2 && k < a_n) { i = k; is_v = false; return true; }
                const int j = k - (a_n > 1 ? 2 : 1);  // V0 K2 V1 K3 ...
                if (j < 2 * (a_n - 2)) { i = (j & 1) ? 2 + j / 2 : j / 2; is_v = !(j & 1); return true; }
                i = a_n - (2 * a_n - k);
                is_v = true;
                return true;
            };
            auto issue = [&] {
                int i;
                bool is_v;
                if (a_next(i, is_v)) {
                    const int tok0 = (aw.t0 + i) * kT, tokens = aw.prefix + aw.nodes;
                    const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.v : p.k) + c * 16;
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const int r = r0 + k * kStep;
                        const bool there = tok0 + r < tokens;
                        const long long row = there ? tree_row(p.at, aw.e, aw.h, tok0 + r) : 0;
                        cp_async16_zfill(raw + a_slot * C::kRawBytes + k * 4096, src + row * D, there);
                    }
                }
                cp_async_commit();
                if (++a_slot == C::kRaw) a_slot = 0;
            };
#pragma unroll
            for (int k = 0; k < C::kRaw - 1; ++k) issue();
            int slot = 0;
            bool ok = true;
            while (ok && next_piece(p, cur, u, end, w)) {
                const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
                if (rows <= 0) continue;
                bool first = true;
                ok = ring_order<MT>(w.t1 - w.t0, [&](int, bool) {
                    issue();
                    if (first) {
                        first = false;
                        if (!wait(q_empty, q_ph)) return false;
                        q_ph ^= 1;
                        const int qc = tid % kChunks, qr = tid / kChunks;
                        for (int b = 0; b < MT; ++b)
#pragma unroll 4
                            for (int k = 0; k < kT * kChunks / 256; ++k) {
                                const int r = qr + k * (256 / kChunks), row = b * kT + r;
                                uint4 x = make_uint4(0, 0, 0, 0);
                                if (row < rows)
                                    x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                                        q_offset(p, w.e, w.h, row0 + row, D) + qc * 8);
                                *reinterpret_cast<uint4*>(smem + b * kT * D * 2 + tile_at(r, qc)) = x;
                            }
                    }
                    if (!wait(empty + ring.i, ring.ph ^ 1)) return false;
                    cp_async_wait<C::kRaw - 1>();
                    uint8_t* dst = smem + C::oStage + ring.i * C::kStage;
#pragma unroll
                    for (int k = 0; k < kMine; ++k) {
                        const int r = r0 + k * kStep;
                        const uint4 x = *reinterpret_cast<const uint4*>(raw + slot * C::kRawBytes + k * 4096);
                        const uint2 a = widen4(x.x), b = widen4(x.y), d = widen4(x.z), f = widen4(x.w);
                        *reinterpret_cast<uint4*>(dst + tile_at(r, 2 * c)) = make_uint4(a.x, a.y, b.x, b.y);
                        *reinterpret_cast<uint4*>(dst + tile_at(r, 2 * c + 1)) = make_uint4(d.x, d.y, f.x, f.y);
                    }
                    proxy_fence();
                    mbar_arrive(full + ring.i);
                    ring.next();
                    if (++slot == C::kRaw) slot = 0;
                    return true;
                });
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp == 8) {
        // ----------------------------------------------------------- products
        Ring<NS> ring;
        uint32_t p_ph[2] = {0, 0};
        constexpr uint32_t kS = instr_desc(kT, false), kO = instr_desc(D, true);
        const uint32_t q_addr = smem_u32(smem), st_addr = smem_u32(smem + C::oStage);
        auto s_of = [&](int s) { return tmem + s * kT; };
        auto o_of = [&](int s) { return tmem + 2 * kT + s * D; };
        auto ready = [&](const Ring<NS>& r) {
            if (!wait(full + r.i, r.ph)) return false;
            proxy_fence();  // the copies' writes, before the products read them
            return true;
        };
        auto scores = [&](int s, int stage) {  // S = Q K^T of stream s
            const uint32_t a = q_addr + (MT == 2 ? s : 0) * kT * D * 2, b = st_addr + stage * C::kStage;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * (kT * 128) + (k & 3) * 32;
                mma_ss(s_of(s), smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), kS, k > 0);
            }
            tc_commit(s_full + s);
        };
        auto values = [&](int s, int stage, bool add) {  // O += P V of stream s
            const uint32_t b = st_addr + stage * C::kStage;
#pragma unroll
            for (int k = 0; k < kT / 16; ++k)
                mma_ts(o_of(s), s_of(s) + k * 8, smem_desc(b + k * 2048, kT * 128, 1024), kO, add || k > 0);
            tc_commit(o_done + s);
        };
        auto weights = [&](int s) {  // P of stream s is there
            if (!wait(p_full + s, p_ph[s])) return false;
            p_ph[s] ^= 1;
            tc_fence_after();
            return true;
        };
        while (next_piece(p, cur, u, end, w)) {
            if (w.nodes * p.G - w.mt * p.tile_rows <= 0) continue;
            const int n = w.t1 - w.t0;
            bool ok = true;
            if (lane == 0) {
                if (MT == 1) {
                    for (int i = 0; ok && i < n && i < 2; ++i) {
                        ok = ready(ring);
                        if (!ok) break;
                        scores(i, ring.i);
                        tc_commit(empty + ring.i);
                        if (i + 1 == n) tc_commit(q_empty);
                        ring.next();
                    }
                    for (int i = 0; ok && i < n; ++i) {
                        const int s = i & 1;
                        ok = ready(ring) && weights(s);
                        if (!ok) break;
                        values(s, ring.i, i >= 2);
                        tc_commit(empty + ring.i);
                        ring.next();
                        if (i + 2 < n) {
                            ok = ready(ring);
                            if (!ok) break;
                            scores(s, ring.i);
                            tc_commit(empty + ring.i);
                            if (i + 3 == n) tc_commit(q_empty);
                            ring.next();
                        }
                    }
                } else {
                    ok = ready(ring);
                    if (ok) {
                        scores(0, ring.i);
                        scores(1, ring.i);
                        tc_commit(empty + ring.i);
                        if (n == 1) tc_commit(q_empty);
                        ring.next();
                    }
                    for (int i = 0; ok && i < n; ++i) {
                        const Ring<NS> rv = ring;
                        ring.next();
                        const bool more = i + 1 < n;
                        ok = ready(rv) && weights(0);
                        if (!ok) break;
                        values(0, rv.i, i > 0);
                        if (more) {
                            ok = ready(ring);
                            if (!ok) break;
                            scores(0, ring.i);
                        }
                        ok = weights(1);
                        if (!ok) break;
                        values(1, rv.i, i > 0);
                        tc_commit(empty + rv.i);
                        if (more) {
                            scores(1, ring.i);
                            tc_commit(empty + ring.i);
                            if (i + 2 == n) tc_commit(q_empty);
                            ring.next();
                        }
                    }
                }
                if (!ok) {  // products in flight end before the tensor memory is given back
                    tc_commit(drain);
                    mbar_wait_bounded(drain, 0, p.err, 3, 10000000ull);
                }
            }
            __syncwarp();
            if (__shfl_sync(0xffffffffu, (int)ok, 0) == 0) break;
        }
    } else {
        // ------------------------------------------------------------ softmax
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
            for (int i = MT == 1 ? st : 0; i < n; i += MT == 1 ? 2 : 1) {
                const int tok0 = (w.t0 + i) * kT;
                const bool masked = tok0 + kT > w.prefix;
                if constexpr (C::kQ8) {  // the tile's scales, ahead of S
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kT / 32; ++k) {
                        const int t = k * 32 + lane;
                        float a = 0.f, b = 0.f;
                        if (tok0 + t < tokens) {
                            const long long row = tree_row(p.at, w.e, w.h, tok0 + t);
                            a = __ldg(p.k_scale + row) * p.qscale;
                            b = __ldg(p.v_scale + row);
                        }
                        ks[t] = a;
                        vs[t] = b;
                    }
                    __syncwarp();
                }
                if (masked) {
                    // values of tree rows that are not finite leave the stage (see the top)
                    const long long use = uses + (MT == 2 ? 2 * i + 1 : n == 1 ? 1 : i < n - 1 ? 2 * i + 2 : 2 * i + 1);
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
                    uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            vis[k] = live ? visible(p, w.e, node, w.nodes, tok0 + 32 * k - w.prefix) : 0u;
                    }
                    // the tile's maximum
                    float mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t x[32];
                        tc_ld32(x, t_s + 32 * k);
                        tc_wait_ld();
                        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float f = __uint_as_float(x[j]);
                            if constexpr (C::kQ8) f *= ks[32 * k + j];
                            if (masked) f = (vis[k] >> j & 1) ? f : -INFINITY;
                            a[j & 3] = fmaxf(a[j & 3], f);
                        }
                        mx = fmaxf(mx, fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])));
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
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t x[32], y[16];
                        tc_ld32(x, t_s + 32 * k);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float f = __uint_as_float(x[j]);
                            float e = ex2(C::kQ8 ? fmaf(f, ks[32 * k + j], base) : fmaf(f, p.qscale, base));
                            if (masked) e = (vis[k] >> j & 1) ? e : 0.f;
                            sum[j & 3] += e;
                            if constexpr (C::kQ8) {
                                e *= vs[32 * k + j];
                                if (masked) e = (vis[k] >> j & 1) ? e : 0.f;
                            }
                            x[j] = __float_as_uint(e);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            y[j] = pack_bf16x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                        tc_st16(t_s + 16 * k, y);
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
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    float f;
                                    if constexpr (C::kQ8) {
                                        const uint8_t code = static_cast<const uint8_t*>(p.v)[row * D + col + j];
                                        f = (code & 0x7f) == 0x7f ? NAN : 0.f;
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
