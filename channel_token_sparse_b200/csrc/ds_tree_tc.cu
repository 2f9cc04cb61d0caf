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
// issues the products, warp 9 brings K and V tiles into a ring of
// 128-byte-swizzled stages by tensor copies (any page size), warps 10 and 11
// the queries. 8-bit tiles land in slots of their own and warps 12 to 19 widen
// them to bf16 (exact) into the ring; their rows' scales multiply S and P.
//
// Measured on a B200: 16 nodes x 4 heads over 4 x 32K bf16 107 us (77 % of the
// copy rate; MT = 1; 8-bit 132), 64 nodes x 4 heads over 128K bf16 176 us (780
// TFLOP/s; MT = 2; 8-bit 252). What bounds MT = 2 is the chain of a stream's tile:
// softmax, PV, S and the wake-ups between them (tensor pipe and special-function
// unit both half busy).
//
// P is rounded to bf16 (2^-9 of a weight at most, each its own way), which is what
// the products take; a second product for the remainders would double P V.
//
// The products take every row of V with every weight, and 0 * NaN is NaN, so
// the softmax warps tidy a tile that reaches past the prefix: rows past the
// sequence become zeros, and the rows of tree nodes (which some query rows may
// not see) are looked through for values that are not finite, which are zeroed
// and added to the rows that do see them at the end. An 8-bit tree row whose
// scales are not finite is set aside the same way.
#include "ds_tree_tc.cuh"

namespace ds {

namespace {

template <int TYPE, int D, int MT>
struct Cfg {
    static constexpr bool kQ8 = TYPE == kTreeE4M3;
    static constexpr int kThreads = kQ8 ? 640 : 384;
    // Registers of a thread by role: 384 (8-bit: 640) threads are launched with
    // 168 (96) each, and the four-warp groups redistribute them: their sums are
    // 208 + 208 + 88 = 3 * 168 and 152 + 152 + 64 + 2 * 56 = 5 * 96.
    static constexpr int kRegSoftmax = kQ8 ? 152 : 208, kRegMma = kQ8 ? 64 : 88, kRegWiden = 56;
    static_assert(kQ8 ? 2 * kRegSoftmax + kRegMma + 2 * kRegWiden <= 5 * 96 : 2 * kRegSoftmax + kRegMma <= 3 * 168, "");
    static constexpr int kStage = kT * D * 2;       // bytes of a K or V tile in bf16
    static constexpr int kQ = MT * kT * D * 2;
    static constexpr int kRaw = kQ8 ? (D == 128 && MT == 2 ? 2 : 4) : 0, kRawBytes = kT * 128;  // slots of 8-bit tiles
    static constexpr int kScale = kQ8 ? 8 * 2 * kT * 4 : 0;  // a softmax warp's K and V scales of a tile
    static constexpr int kStages = D == 128 ? (kQ8 ? 3 : 7 - MT) : 13 - MT - 4 * kQ8;
    static constexpr int oStage = kQ, oRaw = oStage + kStages * kStage, oScale = oRaw + kRaw * kRawBytes;
    static constexpr int oMl = oScale + kScale;             // [2][128] maxima, [2][128] sums
    static constexpr int oBar = oMl + 4 * kT * 4;
    static constexpr int kBars = 2 * kStages + 2 * kRaw + 10;
    static constexpr int kSmem = oBar + kBars * 8 + 64;
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

// The order in which a piece of n token tiles uses the ring, and the use that
// holds V of a tile. MT = 1: K0 K1, then V_i K_{i+2}; MT = 2: K_i V_i.
template <int MT> struct TcOrder {
    static __device__ __forceinline__ RingUse use(int k, int n) {
        if (MT == 2) return RingUse{k >> 1, (k & 1) != 0};
        const int lead = n > 1 ? 2 : 1, j = k - lead;
        if (j < 0) return RingUse{k, false};
        if (j < 2 * (n - 2)) return RingUse{(j & 1) ? 2 + j / 2 : j / 2, (j & 1) == 0};
        return RingUse{k - n, true};  // the last V tiles
    }
    static __device__ __forceinline__ int v_use(int i, int n) {
        return MT == 2 ? 2 * i + 1 : n == 1 ? 1 : i < n - 1 ? 2 * i + 2 : 2 * i + 1;
    }
};

// -------------------------------------------------------------------- kernel

template <int TYPE, int D, int MT>
__global__ void __launch_bounds__(Cfg<TYPE, D, MT>::kThreads, 1) ds_tree_tc_kernel(
    const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
    using C = Cfg<TYPE, D, MT>;
    constexpr int NS = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* ml = reinterpret_cast<float*>(smem + C::oMl);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::oBar);
    uint64_t* empty = full + NS;
    uint64_t* s_full = empty + NS;   // [2] S of a stream is there
    uint64_t* p_full = s_full + 2;   // [2] its P is, and O is ready to take it
    uint64_t* o_done = p_full + 2;   // [2] O has taken it
    uint64_t* q_empty = o_done + 2;  // the piece's S products are done
    uint64_t* q_full = q_empty + 1;  // its queries are there
    uint64_t* xch = q_full + 1;      // softmax warps among themselves
    uint64_t* drain = xch + 1;
    uint64_t* raw_full = drain + 1;  // [kRaw] 8-bit tiles
    uint64_t* raw_empty = raw_full + C::kRaw;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(raw_empty + C::kRaw);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* bad = tmem_slot + 2;   // [8] nodes whose V row holds values that are not finite

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, C::kQ8 ? 4 : 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(raw_full + i, 1);
            mbar_init(raw_empty + i, 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full + s, 1);
            mbar_init(p_full + s, 4);
            mbar_init(o_done + s, 1);
        }
        mbar_init(q_empty, 1);
        mbar_init(q_full, 2);
        mbar_init(xch, 8);
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
        // --------------------------------------------------- widening (8-bit)
        if constexpr (C::kQ8) {
            reg_dec<C::kRegWiden>();
            widen_tiles<D, C::kRaw, NS>(p, smem + C::oRaw, raw_full, raw_empty, smem + C::oStage, full, empty, wait, cur, u,
                                        end, threadIdx.x - 12 * 32);
        }
    } else if (warp >= 8) {
        // -------------------------------------------------- copies, products
        reg_dec<C::kRegMma>();
        if (warp == 9) {
            if constexpr (C::kQ8)
                copy_tiles<TYPE, D, C::kRaw, TcOrder<MT>>(p, &maps.k, &maps.v, smem + C::oRaw, raw_full, raw_empty, wait, cur, u, end);
            else
                copy_tiles<TYPE, D, NS, TcOrder<MT>>(p, &maps.k, &maps.v, smem + C::oStage, full, empty, wait, cur, u, end);
        } else if (warp >= 10) {
            copy_queries<D, MT * kT, C::kQ8>(p, smem, q_full, q_empty, wait, cur, u, end, threadIdx.x - 10 * 32);
        }
        // The products are warp 8's. What their operands and loops depend on comes
        // from votes and reductions, so that it lives in uniform registers: moved
        // there for each instruction, it made a product take 125 cycles to issue.
        const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
        Ring<NS> ring;
        uint32_t p_ph[2] = {0, 0}, q_ph = 0;
        constexpr uint32_t kS = instr_desc(kT, false, false), kO = instr_desc(D, false, true);
        const uint32_t q_addr = smem_u32(smem), st_addr = smem_u32(smem + C::oStage);
        auto s_of = [&](int s) { return tm + s * kT; };
        auto o_of = [&](int s) { return tm + 2 * kT + s * D; };
        auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        auto ready = [&](const Ring<NS>& r) { return all_wait(full + r.i, r.ph); };
        auto commit = [&](uint64_t* bar) { if (elected()) tc_commit(bar); };
        auto scores = [&](int s, int stage) {  // S = Q K^T of stream s
            const uint32_t d = s_of(s);
            const uint64_t a = smem_desc(q_addr + (MT == 2 ? s : 0) * kT * D * 2, 16, 1024);
            const uint64_t b = smem_desc(st_addr + stage * C::kStage, 16, 1024);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * (kT * 128) + (k & 3) * 32) >> 4;
                mma_ss(d, a, off, b, off, kS, k > 0);
            }
            commit(s_full + s);
        };
        auto values = [&](int s, int stage, bool add) {  // O += P V of stream s
            const uint32_t d = o_of(s), a = s_of(s);
            const uint64_t b = smem_desc(st_addr + stage * C::kStage, kT * 128, 1024);
#pragma unroll
            for (int k = 0; k < kT / 16; ++k) mma_ts(d, a + k * 8, b, k * 128, kO, add || k > 0);
            commit(o_done + s);
        };
        auto weights = [&](int s) {  // P of stream s is there
            if (!all_wait(p_full + s, p_ph[s])) return false;
            p_ph[s] ^= 1;
            tc_fence_after();
            return true;
        };
        while (warp == 8) {
            const bool any = next_piece(p, cur, u, end, w);
            if (!__any_sync(0xffffffffu, any)) break;
            if (!__any_sync(0xffffffffu, w.nodes * p.G - w.mt * p.tile_rows > 0)) continue;
            const int n = (int)__reduce_max_sync(0xffffffffu, (unsigned)(w.t1 - w.t0));
            bool ok = all_wait(q_full, q_ph);
            q_ph ^= 1;
            if (MT == 1) {
                // S of the first two tiles, then PV of tile i and S of tile i + 2
                for (int i = -2; ok && i < n; ++i) {
                    const Ring<NS> rv = ring;
                    if (i >= 0) ring.next();
                    // both tiles first: they are there long before the weights
                    ok = (i < 0 || ready(rv)) && (i + 2 >= n || ready(ring));
                    if (ok && i >= 0) {
                        ok = weights(i & 1);
                        if (!ok) break;
                        values(i & 1, rv.i, (i >> 1) % kSpan > 0);
                        commit(empty + rv.i);
                    }
                    if (ok && i + 2 < n) {
                        scores(i & 1, ring.i);
                        commit(empty + ring.i);
                        if (i + 3 == n) commit(q_empty);
                        ring.next();
                    }
                }
            } else {
                // of each stream: PV of tile i, then S of tile i + 1
                Ring<NS> rv = ring;
                for (int i = -1; i < n; ++i) {
                    const bool more = i + 1 < n;
                    if (i >= 0) { rv = ring; ring.next(); }
                    // both tiles first: they are there long before the weights
                    ok = (i < 0 || ready(rv)) && (!more || ready(ring));
                    if (!ok) break;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (i >= 0) {
                            ok = weights(s);
                            if (!ok) break;
                            values(s, rv.i, i % kSpan > 0);
                        }
                        if (more) scores(s, ring.i);
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
        unsigned uses = 0;                          // ring uses of the pieces before
        bool ok = true;
        // This row's second sums (see kSpan), in the workspace: four channels of 128 rows
        // side by side. They are relative to the maximum of their last addition, which
        // stands in ml until the piece's end.
        float4* sums = reinterpret_cast<float4*>(p.sums) + ((size_t)blockIdx.x * 2 + st) * (kT * D / 4) + r;
        auto add_sums = [&](float m, bool both, bool back) {  // the sums (or, back, O) = O (+ the sums)
            const float last = ml[st * kT + r], f = both && last != -INFINITY ? ex2(last - m) : 0.f;
            if (!back) ml[st * kT + r] = m;
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                uint32_t y[32];
                tc_ld(y, t_o + st * D + 32 * k);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float4* at = sums + (8 * k + j / 4) * kT;
                    float4 o = make_float4(__uint_as_float(y[j]), __uint_as_float(y[j + 1]), __uint_as_float(y[j + 2]),
                                           __uint_as_float(y[j + 3]));
                    if (both) {
                        const float4 b = *at;
                        o.x = fmaf(b.x, f, o.x); o.y = fmaf(b.y, f, o.y);
                        o.z = fmaf(b.z, f, o.z); o.w = fmaf(b.w, f, o.w);
                    }
                    if (!back) *at = o;
                    y[j] = __float_as_uint(o.x); y[j + 1] = __float_as_uint(o.y);
                    y[j + 2] = __float_as_uint(o.z); y[j + 3] = __float_as_uint(o.w);
                }
                if (back) tc_st(t_o + st * D + 32 * k, y);
            }
            if (back) tc_wait_st();
        };
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
            for (int i = i0; ok && i < n;) {
                for (const int span = min(n, i + kEvery * kSpan); i < span; i += kEvery) {
                    const int tok0 = (w.t0 + i) * kT;
                    const bool masked = tok0 + kT > w.prefix;
                    if constexpr (C::kQ8) {  // the tile's scales; those of the stream's next tile are read meanwhile
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < kT / 32; ++k) {
                            const int j = tok0 + k * 32 + lane - w.prefix;
                            float a = sc_k[k] * p.qscale, b = sc_v[k];
                            if (!(isfinite(a) && isfinite(b))) {
                                if (j < 0) {  // an infinite key scale makes the scores NaN
                                    a = fmaf(a, 0.f, a);
                                } else {  // not seen by all rows: set aside
                                    a = b = 0.f;
                                    atomicOr(bad + (j >> 5), 1u << (j & 31));
                                }
                            }
                            ks[k * 32 + lane] = a;
                            vs[k * 32 + lane] = b;
                        }
                        __syncwarp();
                    }
                    ok = all_wait(s_full + st, s_ph);
                    if (!ok) break;
                    s_ph ^= 1;
                    if (masked && !C::kQ8) {
                        // The V stage is tidied before the products read it (see the top). Only now:
                        // while S was not there, the stage's use before could still be landing, and
                        // the parity of this one's phase would be that of two before.
                        const unsigned use = uses + TcOrder<MT>::v_use(i, n), stage = use % NS;
                        ok = all_wait(full + stage, use / NS & 1);
                        if (!ok) break;
                        tidy_values<D>(smem + C::oStage + stage * C::kStage, max(w.prefix - tok0, 0), min(tokens - tok0, kT),
                                       tok0 - w.prefix, bad, threadIdx.x & 127);
                        proxy_fence();
                    }
                    tc_fence_after();
                    if (warp_live) {
                        if (masked) {  // what a row does not see gets the score -infinity
#pragma unroll 1
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t vis = live ? visible(p, w.e, node, w.nodes, tok0 + 32 * k - w.prefix) : 0u;
                                uint32_t x[32];
                                tc_ld(x, t_s + 32 * k);
                                tc_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j) {
                                    float f = __uint_as_float(x[j]);
                                    if constexpr (C::kQ8) f *= ks[32 * k + j];
                                    x[j] = (vis >> j & 1) ? __float_as_uint(f) : 0xff800000u;
                                }
                                tc_st(t_s + 32 * k, x);
                            }
                            tc_wait_st();
                            if constexpr (C::kQ8) {  // the scales are in these scores
                                __syncwarp();
                                for (int k = lane; k < kT; k += 32) ks[k] = 1.f;
                                __syncwarp();
                            }
                        }
                        // The tile's maximum. MT = 2, where the softmax is on the critical path:
                        // the scores stay in registers from here on (64 nodes over 128K 177 us
                        // or 185, for all that 250 bytes a thread are spilled; one row block of
                        // 64 rows 117 us so, or 108); else they are read once more.
                        constexpr int kHeld = C::kQ8 || MT == 1 ? 2 : 4;
                        uint32_t x[kHeld][32];
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int k = 0; k < 4; k += kHeld) {
#pragma unroll
                            for (int h = 0; h < kHeld; ++h) tc_ld(x[h], t_s + 32 * (k + h));
                            tc_wait_ld();
                            float a[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int h = 0; h < kHeld; ++h) {
#pragma unroll
                                for (int j = 0; j < 32; j += 8) {
                                    float f[8];
#pragma unroll
                                    for (int q = 0; q < 8; ++q) f[q] = __uint_as_float(x[h][j + q]);
                                    if constexpr (C::kQ8) {
                                        const float4 s0 = *reinterpret_cast<const float4*>(ks + 32 * (k + h) + j);
                                        const float4 s1 = *reinterpret_cast<const float4*>(ks + 32 * (k + h) + j + 4);
                                        f[0] *= s0.x; f[1] *= s0.y; f[2] *= s0.z; f[3] *= s0.w;
                                        f[4] *= s1.x; f[5] *= s1.y; f[6] *= s1.z; f[7] *= s1.w;
                                    }
#pragma unroll
                                    for (int q = 0; q < 4; ++q) a[q] = fmaxf(fmaxf(a[q], f[2 * q]), f[2 * q + 1]);
                                }
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
                                    uint32_t y[32];
                                    tc_ld(y, t_o + st * D + 32 * k);
                                    tc_wait_ld();
#pragma unroll
                                    for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                                    tc_st(t_o + st * D + 32 * k, y);
                                }
                            }
                        }
                        const float base = m == -INFINITY ? 0.f : -m;
                        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                        for (int k = 0; k < 4; k += kHeld) {
                            if constexpr (kHeld < 4) {
#pragma unroll
                                for (int h = 0; h < kHeld; ++h) tc_ld(x[h], t_s + 32 * (k + h));
                                tc_wait_ld();
                            }
#pragma unroll
                            for (int h = 0; h < kHeld; ++h) {
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
                                        fma2(f[0], f[1], p.qscale, base);
                                        fma2(f[2], f[3], p.qscale, base);
                                    }
#pragma unroll
                                    for (int q = 0; q < 4; ++q) f[q] = ex2(f[q]);
                                    add2(sum[0], sum[1], f[0], f[1]);
                                    add2(sum[2], sum[3], f[2], f[3]);
                                    if constexpr (C::kQ8) {
                                        const float4 sc = *reinterpret_cast<const float4*>(vs + 32 * (k + h) + j);
                                        f[0] *= sc.x; f[1] *= sc.y; f[2] *= sc.z; f[3] *= sc.w;
                                    }
                                    y[j / 2] = pack_bf16x2(f[0], f[1]);
                                    y[j / 2 + 1] = pack_bf16x2(f[2], f[3]);
                                }
                                tc_st(t_s + 16 * (k + h), y);
                            }
                        }
                        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        tc_wait_st();
                    }
                    tc_fence_before();
                    warp_arrive(p_full + st);
                    if (C::kQ8 && i + kEvery < n) scales(tok0 + kEvery * kT);
                    ++o_cnt;
                    ++done;
                }
                if (ok && i < n && warp_live) {  // O starts again
                    ok = all_wait(o_done + st, (o_cnt - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    add_sums(m, done > kSpan, false);
                }
            }
            if (!ok) break;
            uses += 2 * n;
            // the piece's result
            if (done > 0) {
                ok = all_wait(o_done + st, (o_cnt - 1) & 1);
                if (!ok) break;
                if (done > kSpan && warp_live) {
                    tc_fence_after();
                    add_sums(m, true, true);
                }
            }
            ml[st * kT + r] = m;
            ml[(2 + st) * kT + r] = l;
            tc_fence_before();
            warp_arrive(xch);
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
                    __syncwarp();
                    tc_ld(x, t_o + (MT == 2 ? st * D : 0) + col);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __uint_as_float(x[j]) * f0;
                    if (MT == 1 && n > 1) {
                        tc_ld(x, t_o + D + col);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(x[j]), f1, o[j]);
                    }
                    if constexpr (C::kQ8) {  // channels back in their order
#pragma unroll
                        for (int j = 1; j < 32; j += 4) {
                            const float y = o[j];
                            o[j] = o[j + 1];
                            o[j + 1] = y;
                        }
                    }
                    if (!live) continue;
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
                if (any_bad && live) {
#pragma unroll 1
                    for (int c = col0; c < col0 + kCols; ++c)
                        add_result(p, whole ? nullptr : part + 2 * p.part_rows,
                                   whole ? at + c : (size_t)item_row * D + c, not_finite_seen<TYPE, D>(p, w, node, bad, c));
                }
            }
            // both streams have read O, the maxima and the marks before either goes on
            tc_fence_before();
            warp_arrive(xch);
            ok = all_wait(xch, x_ph);
            if (!ok) break;
            x_ph ^= 1;
            if (any_bad && threadIdx.x < 8) bad[threadIdx.x] = 0;
            if (any_bad) {  // cleared before the next piece marks
                warp_arrive(xch);
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
cudaError_t run(const TreeParams& p, const TreeMaps& m, cudaStream_t st) {
    using C = Cfg<TYPE, D, MT>;
    cudaError_t e = cudaFuncSetAttribute(ds_tree_tc_kernel<TYPE, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
    ds_tree_tc_kernel<TYPE, D, MT><<<p.grid, C::kThreads, C::kSmem, st>>>(p, m);
    return cudaGetLastError();
}

}  // namespace

// The driver's encoder, fetched through the runtime (the library does not link
// the driver library).
cudaError_t make_tree_maps(const TreeParams& p, int type, int d, TreeMaps* m) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return cudaErrorNotSupported;
    const bool q8 = type == kTreeE4M3;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)p.cache_rows}, stride[1] = {(cuuint64_t)(q8 ? d : 2 * d)};
    const int page = p.at.block_table ? 1 << p.at.page_shift : kT;
    const cuuint32_t box[2] = {(cuuint32_t)(q8 ? 128 : 64), (cuuint32_t)(page < kT ? page : kT)}, one[2] = {1, 1};
    for (int i = 0; i < 2; ++i) {
        const CUresult r = encode(i ? &m->v : &m->k, q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                                  const_cast<void*>(i ? p.v : p.k), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  q8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

TreePlan plan_tree_tc(int rows, int type) {
    // us a call, 4 x 32K tokens of 8 kv heads unless stated. Products with tokens as
    // rows (ds_tree_few.cu) or with queries as rows:
    //   16 rows bf16 100 or 105 (512 tokens 14.8 or 16.6), 8-bit 87 or 130;
    //   20 rows bf16 110 or 105, 8-bit 108 or 130; 32 rows bf16 112 or 106, 8-bit
    //   109 or 130; 28 rows, 16 x 8K bf16 in pages, with the write 91 or 82.
    // One block of 128 rows or two, that share the tiles they read:
    //   128 rows bf16 114 or 146, 8-bit 139 or 192 (two, half of them empty);
    //   132 rows bf16 189 or 160, 8-bit 235 or 209.
    const int few = type == kTreeE4M3 ? 32 : 16;
    const int tile = rows <= 16 ? 16 : rows <= few ? few : rows <= kT ? kT : 2 * kT;
    return TreePlan{tile, kT, 148};
}

size_t tree_tc_sums(const TreePlan& plan, int grid, long long tiles, int d) {
    // tiles of a stream; ds_tree_few.cu has them in tensor memory
    const long long n = plan.tile_rows == 2 * kT ? tiles : (tiles + 1) / 2;
    return plan.tile_rows < kT || n <= kSpan ? 0 : (size_t)grid * 2 * kT * d * sizeof(float);
}

cudaError_t launch_tree_few(const TreeParams& p, const TreeMaps& m, int type, int d, cudaStream_t st);

cudaError_t launch_tree_tc(const TreeParams& p, int type, int d, cudaStream_t st) {
    TreeMaps m;
    const cudaError_t e = make_tree_maps(p, type, d, &m);
    if (e != cudaSuccess) return e;
    if (p.tile_rows < kT) return launch_tree_few(p, m, type, d, st);
    const bool two = p.tile_rows == 2 * kT;
#define DS_T(TY, D_) (two ? run<TY, D_, 2>(p, m, st) : run<TY, D_, 1>(p, m, st))
    if (type == kTreeBF16) return d == 64 ? DS_T(kTreeBF16, 64) : DS_T(kTreeBF16, 128);
    return d == 64 ? DS_T(kTreeE4M3, 64) : DS_T(kTreeE4M3, 128);
#undef DS_T
}

}  // namespace ds
