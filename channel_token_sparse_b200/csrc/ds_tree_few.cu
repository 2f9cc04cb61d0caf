// ds_tree_few.cu -- tree attention of up to 16 (8-bit caches: 32) query rows a kv
// head over bf16 and 8-bit caches, on the tensor cores, for sm_100a.
//
// The products are taken the other way round from ds_tree_tc.cu: S^T = K Q^T
// and O^T += V^T P^T, so that the 128 rows the tensor cores want are the
// tile's tokens (then the channels) and N = 16 or 32 covers the query
// rows. With few rows this is what keeps the kernel at the cache's bandwidth:
// a tile costs N / 128 of the products and of the exponentials, a thread has
// one token and N of them (rather than one row and 128), and an 8-bit row's
// scales are two numbers of its thread. P^T goes to shared memory (a token's
// weights side by side), S^T and O^T live in tensor memory.
//
// Two warpgroups take alternate token tiles, each with its own running
// maxima, sums and O^T, joined at the end of a piece. A tile moves a maximum
// only when one of its scores passes it by 8 (see ds_tree_tc.cu); whether one
// does is the only thing the four warps agree on in every tile. Sums stay a
// thread's own until the end. Measured on a B200: one token of 32 heads over
// 256K 8-bit tokens 502 us (67 % of the copy rate; widening the codes and the
// issue of the products bound it), 8 nodes over 8 x 4K 8-bit 97 us, one token of 8
// heads of 4 over 4 x 128K bf16 329 us (all of the copy rate). Roles, ring, loaders
// and the treatment of values that are not finite in tree rows are those of
// ds_tree_tc.cu.
#include "ds_tree_tc.cuh"

namespace ds {

namespace {

constexpr float kFloor = -3.0e38f;  // a maximum before any token

template <int TYPE, int D, int N>
struct Cfg {
    static constexpr bool kQ8 = TYPE == kTreeE4M3;
    static constexpr int kThreads = kQ8 ? 640 : 384;
    // Registers of a thread by role (see ds_tree_tc.cu): launched with 168
    // (8-bit: 96), 208 + 208 + 88 = 3 * 168 and 152 + 152 + 64 + 2 * 56 = 5 * 96.
    static constexpr int kRegSoftmax = kQ8 ? 152 : 208, kRegMma = kQ8 ? 64 : 88, kRegWiden = 56;
    static_assert(kQ8 ? 2 * kRegSoftmax + kRegMma + 2 * kRegWiden <= 5 * 96 : 2 * kRegSoftmax + kRegMma <= 3 * 168, "");
    static constexpr int kStage = kT * D * 2;
    static constexpr int kStages = D == 128 ? (kQ8 ? 3 : 5) : (kQ8 ? 6 : 10);
    static constexpr int kRaw = kQ8 ? 4 : 0, kRawBytes = kT * 128;  // slots of 8-bit tiles
    static constexpr int kQ = N * D * 2, kP = kT * 128;  // P^T: a token's weights in 128 bytes
    static constexpr int oP = kQ, oStage = oP + 2 * kP, oRaw = oStage + kStages * kStage, oStat = oRaw + kRaw * kRawBytes;
    // floats: maxima [2][N], factors [2][N], partial [2][4][N], result [4][N], maxima of the second O^T [2][N]
    static constexpr int kStat = 18 * N;
    static constexpr int oBar = oStat + kStat * 4;
    static constexpr int kBars = 2 * kStages + 2 * kRaw + 12;
    static constexpr int kSmem = oBar + kBars * 8 + 64;
    static_assert(kSmem <= 227 * 1024 && kQ % 1024 == 0, "shared memory");
    // K_i and V_i are five uses of the ring apart at most: see the tidying
    static_assert(kQ8 || kStages >= 5, "stages");
    static constexpr int kCols = N == 32 ? 256 : 128;  // tensor memory: 4 S^T, 2 O^T and 2 second O^T of N columns
};

// K0 K1, then K_{i+2} V_i.
struct FewOrder {
    static __device__ __forceinline__ RingUse use(int k, int n) {
        const int j = k - 2;
        if (k < 2 && k < n) return RingUse{k, false};
        if (j < 2 * (n - 2)) return RingUse{(j & 1) ? j / 2 : 2 + j / 2, (j & 1) != 0};
        return RingUse{k - n, true};
    }
    static __device__ __forceinline__ int v_use(int i, int n) { return n == 1 ? 1 : i < n - 2 ? 2 * i + 3 : n + i; }
};

// Whether the predicate holds in any of the 128 threads of barrier `id`.
__device__ __forceinline__ bool any_of_group(int id, bool x) {
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
                 " selp.b32 %0, 1, 0, q;\n}" : "=r"(r) : "r"((uint32_t)x), "r"(id) : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// Reduces V values over the warp; lane x ends with that of value x * V / 32.
template <int V, bool MAX> __device__ __forceinline__ float warp_reduce_to_lane(float (&v)[V]) {
#pragma unroll
    for (int step = 0; step < 5; ++step) {
        const int msk = 16 >> step, half = V >> (step + 1);
        if (half > 0) {
            const bool up = (lane_id() & msk) != 0;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float keep = up ? v[i + half] : v[i];
                const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + half], msk);
                v[i] = MAX ? fmaxf(keep, got) : keep + got;
            }
        } else {
            const float got = __shfl_xor_sync(0xffffffffu, v[0], msk);
            v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        }
    }
    return v[0];
}

template <int TYPE, int D, int N>
__global__ void __launch_bounds__(Cfg<TYPE, D, N>::kThreads, 1) ds_tree_few_kernel(
    const __grid_constant__ TreeParams p, const __grid_constant__ TreeMaps maps) {
    using C = Cfg<TYPE, D, N>;
    constexpr int NS = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    float* s_max = reinterpret_cast<float*>(smem + C::oStat);  // [2][N]
    float* s_fac = s_max + 2 * N;                              // [2][N]
    float* s_red = s_fac + 2 * N;                              // [2][4][N]
    float* s_fin = s_red + 8 * N;                              // [4][N]: factors of the two streams, 1 / sum, -
    float* s_last = s_fin + 4 * N;                             // [2][N]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::oBar);
    uint64_t* empty = full + NS;
    uint64_t* s_full = empty + NS;   // [2][2] S^T of a stream's tile is there
    uint64_t* p_full = s_full + 4;   // [2] its P^T is, and O^T is ready to take it
    uint64_t* o_done = p_full + 2;   // [2] O^T has taken it
    uint64_t* q_empty = o_done + 2;  // the piece's S^T products are done
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
        for (int s = 0; s < 4; ++s) mbar_init(s_full + s, 1);
        for (int s = 0; s < 2; ++s) {
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
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "n"(C::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Waiter wait{stop, p.err};
    auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

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
                copy_tiles<TYPE, D, C::kRaw, FewOrder>(p, &maps.k, &maps.v, smem + C::oRaw, raw_full, raw_empty, wait, cur, u, end);
            else
                copy_tiles<TYPE, D, NS, FewOrder>(p, &maps.k, &maps.v, smem + C::oStage, full, empty, wait, cur, u, end);
        } else if (warp >= 10) {
            copy_queries<D, N, C::kQ8>(p, smem, q_full, q_empty, wait, cur, u, end, threadIdx.x - 10 * 32);
        }
        // The products are warp 8's. What their operands and loops depend on comes
        // from votes and reductions, so that it lives in uniform registers: moved
        // there for each instruction, it made a product take 125 cycles to issue.
        const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
        Ring<NS> ring;
        uint32_t p_ph[2] = {0, 0}, q_ph = 0;
        constexpr uint32_t kS = instr_desc(N, false, false), kO = instr_desc(N, true, true);
        const uint32_t q_addr = smem_u32(smem), p_addr = smem_u32(smem + C::oP), st_addr = smem_u32(smem + C::oStage);
        while (warp == 8) {
            const bool more = next_piece(p, cur, u, end, w);
            if (!__any_sync(0xffffffffu, more)) break;
            if (!__any_sync(0xffffffffu, w.nodes * p.G - w.mt * p.tile_rows > 0)) continue;
            const int n = (int)__reduce_max_sync(0xffffffffu, (unsigned)(w.t1 - w.t0));
            bool ok = all_wait(q_full, q_ph);
            q_ph ^= 1;
            // S^T of tile i + 2, then PV of tile i
            for (int i = -2; ok && i < n; ++i) {
                const int s = i & 1;
                if (i + 2 < n) {
                    ok = all_wait(full + ring.i, ring.ph);
                    if (!ok) break;
                    const int b = 2 * s + (((i + 2) >> 1) & 1);
                    const uint32_t d = tm + b * N;
                    const uint64_t ka = smem_desc(st_addr + ring.i * C::kStage, 16, 1024), qb = smem_desc(q_addr, 16, 1024);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(d, ka, ((k >> 2) * (kT * 128) + (k & 3) * 32) >> 4, qb,
                               ((k >> 2) * (N * 128) + (k & 3) * 32) >> 4, kS, k > 0);
                    if (elected()) {
                        tc_commit(s_full + b);
                        tc_commit(empty + ring.i);
                        if (i + 3 == n) tc_commit(q_empty);
                    }
                    ring.next();
                }
                if (i >= 0) {
                    ok = all_wait(full + ring.i, ring.ph) && all_wait(p_full + s, p_ph[s]);
                    if (!ok) break;
                    p_ph[s] ^= 1;
                    tc_fence_after();
                    const uint32_t d = tm + 4 * N + s * N;
                    // (64 channels: the other 64 rows repeat them)
                    const uint64_t va = smem_desc(st_addr + ring.i * C::kStage, D == 128 ? kT * 128 : 0, 1024);
                    const uint64_t pb = smem_desc(p_addr + s * C::kP, 16, 1024);
#pragma unroll
                    for (int k = 0; k < kT / 16; ++k) mma_ss(d, va, k * 128, pb, k * 128, kO, (i >> 1) % kSpan > 0 || k > 0);
                    if (elected()) {
                        tc_commit(o_done + s);
                        tc_commit(empty + ring.i);
                    }
                    ring.next();
                }
            }
            if (!ok) {  // products in flight end before the tensor memory is given back
                if (elected()) tc_commit(drain);
                mbar_wait_bounded(drain, 0, p.err, 3, 10000000ull);
                break;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        reg_inc<C::kRegSoftmax>();
        constexpr int HN = C::kQ8 ? 16 : N, H = N / HN;  // columns a thread holds at a time
        const int st = warp >> 2, bar = 1 + st;         // stream, its barrier
        const int t = threadIdx.x & 127;                // token of a tile; channel of O^T
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + 2 * st * N, t_o = tmem + lanes + 4 * N;
        // Moves O^T into the second one (back: the other way), with the second one before
        // where there is one (see kSpan). That is relative to the maxima of the move before.
        auto move_sums = [&](bool both, bool back) {
            const float *m = s_max + st * N, *last = s_last + st * N;
            const uint32_t o = t_o + st * N, second = o + 2 * N;
#pragma unroll 1
            for (int c0 = 0; c0 < N; c0 += 16) {
                float a[16], b[16];
                load_columns<16>(a, o + c0);
                if (both) {
                    load_columns<16>(b, second + c0);
#pragma unroll
                    for (int c = 0; c < 16; ++c) a[c] = fmaf(b[c], ex2(last[c0 + c] - m[c0 + c]), a[c]);
                }
                store_columns<16>((back ? o : second) + c0, a);
            }
            tc_wait_st();
            group_sync(bar);
            if (t < N) s_last[st * N + t] = m[t];
        };
        uint8_t* pt = smem + C::oP + st * C::kP + t * 128;
        // a wait that the warpgroup leaves with one answer, so that none of its warps waits for one that left
        auto group_wait = [&](uint64_t* b, uint32_t parity) { return !any_of_group(bar, !wait(b, parity)); };
        float *mx = s_max + st * N, *fac = s_fac + st * N, *red = s_red + st * 4 * N;
        uint32_t s_ph[2] = {0, 0}, o_cnt = 0, x_ph = 0;  // o_cnt: products awaited or due on o_done
        unsigned uses = 0;                               // ring uses of the pieces before
        bool ok = true;
        while (next_piece(p, cur, u, end, w)) {
            const int rows = min(w.nodes * p.G - w.mt * p.tile_rows, N);
            if (rows <= 0) continue;
            const int n = w.t1 - w.t0, tokens = w.prefix + w.nodes, row0 = w.mt * p.tile_rows;
            float l[N];
#pragma unroll
            for (int c = 0; c < N; ++c) l[c] = 0.f;
            int done = 0;  // tiles of this stream
            float sc_k = 0.f, sc_v = 0.f;  // 8-bit: scales of this thread's token; 0 past the sequence
            auto scales = [&](int tok) {
                const bool there = tok < tokens;
                const long long row = there ? tree_row(p.at, w.e, w.h, tok) : 0;
                sc_k = there ? __ldg(p.k_scale + row) : 0.f;
                sc_v = there ? __ldg(p.v_scale + row) : 0.f;
            };
            if (C::kQ8 && st < n) scales((w.t0 + st) * kT + t);
            for (int i = st; ok && i < n;) {
                for (const int span = min(n, i + 2 * kSpan); i < span; i += 2) {
                    const int tok0 = (w.t0 + i) * kT, node_t = tok0 + t - w.prefix;  // this token's node (negative: prefix)
                    const bool masked = tok0 + kT > w.prefix;
                    float ks = p.qscale, vs = 1.f;
                    if constexpr (C::kQ8) {
                        ks = sc_k * p.qscale;
                        vs = sc_v;
                        if (!(isfinite(ks) && isfinite(vs))) {
                            if (node_t < 0) {  // an infinite key scale makes the scores NaN
                                ks = fmaf(ks, 0.f, ks);
                            } else {  // not seen by all rows: set aside
                                ks = vs = 0.f;
                                atomicOr(bad + (node_t >> 5), 1u << (node_t & 31));
                            }
                        }
                    }
                    bool fine = true;
                    uint32_t vis = ~0u;  // query rows that see this token
                    if (masked) {
                        if (node_t >= w.nodes) vis = 0;
                        else if (node_t >= 0) {
                            vis = 0;
                            const uint32_t g = (1u << p.G) - 1;
                            for (int r = 0, x = row0 / p.G; r < rows; ++x, r += p.G)
                                if (mask_word(p, w.e, x, node_t >> 5) >> (node_t & 31) & 1) vis |= g << r;
                        }
                    }
                    const int buf = (i >> 1) & 1;
                    fine = all_wait(s_full + 2 * st + buf, s_ph[buf]) && fine;
                    s_ph[buf] ^= 1;
                    if (masked && !C::kQ8) {
                        // The V stage is tidied (see ds_tree_tc.cu). Only now: while S^T was not
                        // there, the stage's use before could still be landing, and the parity
                        // of this one's phase would be that of two before.
                        const unsigned use = uses + FewOrder::v_use(i, n), stage = use % NS;
                        fine = all_wait(full + stage, use / NS & 1) && fine;
                        if (fine)
                            tidy_values<D>(smem + C::oStage + stage * C::kStage, max(w.prefix - tok0, 0),
                                           min(tokens - tok0, kT), tok0 - w.prefix, bad, t);
                    }
                    if (done > 0) fine = all_wait(o_done + st, (o_cnt - 1) & 1) && fine;  // P^T and O^T are free
                    tc_fence_after();
                    float x[HN];
                    auto scores = [&](int h) {
                        load_columns<HN>(x, t_s + buf * N + h * HN);
#pragma unroll
                        for (int c = 0; c < HN; ++c) x[c] *= ks;
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < HN; ++c) x[c] = (vis >> (h * HN + c) & 1) ? x[c] : -INFINITY;
                        }
                    };
                    bool move = done == 0 || !fine;
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        scores(h);
                        if (done > 0) {
                            float top = -INFINITY;
#pragma unroll
                            for (int c = 0; c < HN; c += 4) {
                                const float4 m4 = *reinterpret_cast<const float4*>(mx + h * HN + c);
                                top = fmaxf(fmaxf(top, x[c] - m4.x), x[c + 1] - m4.y);
                                top = fmaxf(fmaxf(top, x[c + 2] - m4.z), x[c + 3] - m4.w);
                            }
                            move = move || top > 8.f;
                        }
                    }
                    if (any_of_group(bar, move)) {
                        if (any_of_group(bar, !fine)) { ok = false; break; }
                        // the tile's maxima, over 32 tokens and then over the four warps
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            if (H > 1) scores(h);
                            float y[HN];
#pragma unroll
                            for (int c = 0; c < HN; ++c) y[c] = x[c];
                            const float top = warp_reduce_to_lane<HN, true>(y);
                            if (lane % (32 / HN) == 0) red[(warp & 3) * N + h * HN + lane / (32 / HN)] = top;
                        }
                        group_sync(bar);
                        if (t < N) {
                            const float top = fmaxf(fmaxf(red[t], red[N + t]), fmaxf(red[2 * N + t], red[3 * N + t]));
                            const float old = done > 0 ? mx[t] : kFloor;
                            const float now = done == 0 || top > old + 8.f ? fmaxf(top, old) : old;
                            fac[t] = ex2(old - now);
                            mx[t] = now;
                        }
                        group_sync(bar);
                        if (done > 0) {
#pragma unroll
                            for (int h = 0; h < H; ++h) {
                                float y[HN];
                                load_columns<HN>(y, t_o + st * N + h * HN);
#pragma unroll
                                for (int c = 0; c < HN; ++c) {
                                    const float f = fac[h * HN + c];
                                    y[c] *= f;
                                    l[h * HN + c] *= f;
                                }
                                store_columns<HN>(t_o + st * N + h * HN, y);
                            }
                            tc_wait_st();
                        }
                    }
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        if (H > 1) scores(h);
#pragma unroll
                        for (int c = 0; c < HN; c += 8) {
                            const float4 a = *reinterpret_cast<const float4*>(mx + h * HN + c);
                            const float4 b = *reinterpret_cast<const float4*>(mx + h * HN + c + 4);
                            float e[8] = {x[c] - a.x, x[c + 1] - a.y, x[c + 2] - a.z, x[c + 3] - a.w,
                                          x[c + 4] - b.x, x[c + 5] - b.y, x[c + 6] - b.z, x[c + 7] - b.w};
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                e[k] = ex2(e[k]);
                                l[h * HN + c + k] += e[k];
                                if constexpr (C::kQ8) e[k] *= vs;
                            }
                            const uint4 y = make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]),
                                                       pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7]));
                            *reinterpret_cast<uint4*>(pt + ((((h * HN + c) >> 3) ^ (t & 7)) << 4)) = y;
                        }
                    }
                    proxy_fence();
                    tc_fence_before();
                    warp_arrive(p_full + st);
                    if (C::kQ8 && i + 2 < n) scales(tok0 + 2 * kT + t);  // (before, the fence would wait for them)
                    ++o_cnt;
                    ++done;
                }
                if (ok && i < n) {  // O^T starts again
                    ok = group_wait(o_done + st, (o_cnt - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    move_sums(done > kSpan, false);
                }
            }
            if (!ok) break;
            uses += 2 * n;
            // the piece's result: maxima and sums of both streams first
            if (done > 0) {
                ok = group_wait(o_done + st, (o_cnt - 1) & 1);
                if (!ok) break;
                if (done > kSpan) {
                    tc_fence_after();
                    move_sums(true, true);
                }
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float y[HN];
#pragma unroll
                for (int c = 0; c < HN; ++c) y[c] = l[h * HN + c];
                const float sum = warp_reduce_to_lane<HN, false>(y);
                if (lane % (32 / HN) == 0) red[(warp & 3) * N + h * HN + lane / (32 / HN)] = sum;
            }
            if (done == 0 && t < N) mx[t] = kFloor;
            tc_fence_before();
            warp_arrive(xch);
            ok = group_wait(xch, x_ph);
            if (!ok) break;
            x_ph ^= 1;
            tc_fence_after();
            uint32_t any_bad = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) any_bad |= bad[k];
            const bool whole = w.whole();
            float* part = part_of(p, blockIdx.x, w.t0 == 0, D);
            if (t < N / 2) {  // the rows that this warpgroup will write
                const int r = st * (N / 2) + t;
                const float m0 = s_max[r], m1 = s_max[N + r], mm = fmaxf(m0, m1);
                const float f0 = ex2(m0 - mm), f1 = ex2(m1 - mm);
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) sum += s_red[k * N + r] * f0 + s_red[(4 + k) * N + r] * f1;
                s_fin[r] = f0;
                s_fin[N + r] = f1;
                s_fin[2 * N + r] = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                if (!whole && r < rows) {
                    part[r] = mm;
                    part[p.part_rows + r] = sum;
                }
            }
            warp_arrive(xch);
            ok = group_wait(xch, x_ph);
            if (!ok) break;
            x_ph ^= 1;
            // a thread has one channel of O^T, and half of the rows
            const int first = st * (N / 2), ch = C::kQ8 ? widened_channel(t) : t;
            constexpr int kG = N / 2 < 16 ? N / 2 : 16;
            const int warp_c = (warp & 3) * 32;
            if (warp_c < D) {
#pragma unroll 1
                for (int g = first; g < min(first + N / 2, rows); g += kG) {
                    float a[kG], b[kG];
                    load_columns<kG>(a, t_o + g);
                    if (n > 1) load_columns<kG>(b, t_o + N + g);
#pragma unroll
                    for (int c = 0; c < kG; ++c) {
                        const int r = g + c;
                        if (r >= rows) break;
                        float o = a[c] * s_fin[r];
                        if (n > 1) o = fmaf(b[c], s_fin[N + r], o);
                        o *= s_fin[2 * N + r];
                        if (!whole) {
                            part[2 * p.part_rows + (size_t)r * D + ch] = o;
                        } else {
                            const size_t at = q_offset(p, w.e, w.h, row0 + r, D) + ch;
                            if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
                            else static_cast<float*>(p.out)[at] = o;
                        }
                    }
                }
            }
            if (any_bad && warp_c < D) {
#pragma unroll 1
                for (int r = first; r < min(first + N / 2, rows); ++r) {
                    const float f = not_finite_seen<TYPE, D>(p, w, (row0 + r) / p.G, bad, ch);
                    add_result(p, whole ? nullptr : part + 2 * p.part_rows,
                               whole ? q_offset(p, w.e, w.h, row0 + r, D) + ch : (size_t)r * D + ch, f);
                }
            }
            // both streams have read O^T, the statistics and the marks before either goes on
            tc_fence_before();
            warp_arrive(xch);
            ok = group_wait(xch, x_ph);
            if (!ok) break;
            x_ph ^= 1;
            if (any_bad) {  // cleared before the next piece marks
                if (threadIdx.x < 8) bad[threadIdx.x] = 0;
                warp_arrive(xch);
                ok = group_wait(xch, x_ph);
                if (!ok) break;
                x_ph ^= 1;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kCols) : "memory");
    }
}

template <int TYPE, int D, int N>
cudaError_t run(const TreeParams& p, const TreeMaps& m, cudaStream_t st) {
    using C = Cfg<TYPE, D, N>;
    cudaError_t e = cudaFuncSetAttribute(ds_tree_few_kernel<TYPE, D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmem);
    if (e != cudaSuccess) return e;
    ds_tree_few_kernel<TYPE, D, N><<<p.grid, C::kThreads, C::kSmem, st>>>(p, m);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_few(const TreeParams& p, const TreeMaps& m, int type, int d, cudaStream_t st) {
    if (type == kTreeBF16) return d == 64 ? run<kTreeBF16, 64, 16>(p, m, st) : run<kTreeBF16, 128, 16>(p, m, st);
    if (p.tile_rows == 16) return d == 64 ? run<kTreeE4M3, 64, 16>(p, m, st) : run<kTreeE4M3, 128, 16>(p, m, st);
    return d == 64 ? run<kTreeE4M3, 64, 32>(p, m, st) : run<kTreeE4M3, 128, 32>(p, m, st);
}

}  // namespace ds
