// ds_tree_tc.cuh -- what the tensor-core kernels of the tree attention share:
// tcgen05 wrappers, bounded waits, the ring of K and V stages and its loaders.
#pragma once

#include <cuda.h>
#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kT = 128;  // tokens of a tile, and rows of a row block

// The tensor cores cut off, rather than round, what a product adds to an
// accumulator, so a long sum falls behind: by 1.2e-4 of itself after 256 tiles of
// values of one sign, 1.9 % after 32K of them (4M tokens). So after kSpan tiles of
// a stream its O goes into a second accumulator by rounded additions and starts
// again: 6e-5 at most. Pieces of so many tiles are long ones; short ones do not pay.
constexpr int kSpan = kTreeSpan;

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
// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}
// One product of 16 k-values; A and B by the low words of their descriptors
// (the high words do not change with the address). Every one elects its lane:
// with the products in one elected branch, or with 64-bit descriptor sums, a
// product takes 47 to 77 cycles to issue, so 40 (N = 16) or 64 (N = 128).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint32_t a_off, uint64_t b, uint32_t b_off, uint32_t idesc,
                                       bool add) {
    if (elected())
        asm volatile("{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %6, 0;\n mov.b64 a, {%1, %2};\n"
                     " mov.b64 b, {%3, %4};\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}"
                     ::"r"(d), "r"((uint32_t)a + a_off), "r"((uint32_t)(a >> 32)), "r"((uint32_t)b + b_off),
                       "r"((uint32_t)(b >> 32)), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t b_off, uint32_t idesc, bool add) {
    if (elected())
        asm volatile("{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.u32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}"
                     ::"r"(d), "r"(a), "r"((uint32_t)b + b_off), "r"((uint32_t)(b >> 32)), "r"(idesc),
                       "r"((uint32_t)add) : "memory");
}
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// (x, y) = (x, y) * a + b, and (x, y) += (a, b), two at a time.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b) {
    asm("{\n .reg .b64 u, v, w;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %2};\n mov.b64 w, {%3, %3};\n"
        " fma.rn.f32x2 u, u, v, w;\n mov.b64 {%0, %1}, u;\n}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    asm("{\n .reg .b64 u, v;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n"
        " add.rn.f32x2 u, u, v;\n mov.b64 {%0, %1}, u;\n}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}

// ------------------------------------------------------------------- waiting

// A wait gives up after about a second, or when another one of the CTA did:
// every role then leaves its loop (see mbar_wait_bounded). That is far more than
// a tile takes. The wait for a whole piece (2^24 tiles at most) has a limit of
// ten minutes: whatever a piece could hang on is waited for by another role,
// whose second ends this wait too.
constexpr uint64_t kTileWait = 1000000000ull, kPieceWait = 600 * kTileWait;
struct Waiter {
    volatile int* stop;
    unsigned int* err;
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, uint64_t limit = kTileWait) const {
        return mbar_try_wait(bar, parity) || poll(bar, parity, limit);
    }
    __device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity, uint64_t limit) const {
        const uint64_t t0 = global_ns();
        for (;;) {
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*stop) return false;
            if (global_ns() - t0 > limit) break;
        }
        *stop = 1;
        note_timeout(err, 3);
        return false;
    }
};

// One arrival for the warp, after all its lanes' work (an arrival of every lane
// is serialised: 256 of them a tile took longer than the tile).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(bar);
}

// A place in the ring of stages: consecutive uses of stage `i`, phase `ph`.
template <int N> struct Ring {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() { if (++i == N) { i = 0; ph ^= 1; } }
};

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

// Four e4m3 codes c0 .. c3 -> bf16 pairs (c0, c2) and (c1, c3), exact. A code's
// sign, exponent and mantissa bits at their places in a bf16 are its value
// times 2^-120 (the difference of the exponents' biases, subnormals too); the
// product with 2^120 is exact. The even codes get there by multiplications (the
// sign, 16 times too low then, by 240 more), the odd ones by shifts and masks:
// the conversion instructions, and then the logic unit alone, bounded 8-bit
// tiles. So within four channels the second and third change places, which the
// queries and the output make good. The NaN code becomes +-480: rows that are
// not finite are marked by their scale.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    uint32_t a = (w & 0x00800080u) * 240u + (w & 0x00ff00ffu) * 16u;
    uint32_t b = (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(0x7b807b80u));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(0x7b807b80u));
    return make_uint2(a, b);
}
// The channel at place c of a widened row, and the place of channel c.
__device__ __forceinline__ constexpr int widened_channel(int c) { return (c & ~3) | (c & 1) << 1 | (c >> 1 & 1); }

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

// Tidies rows [b, 128) of a bf16 V stage before the products read it: zeroes
// the values that are not finite in the tile's tree rows [b, have) and marks
// their nodes (row 0 is node `node0`, negative in the prefix), and clears the
// rows past the sequence. Thread t of 128.
template <int D>
__device__ __forceinline__ void tidy_values(uint8_t* v, int b, int have, int node0, uint32_t* bad, int t) {
    constexpr int kChunks = D / 8;
    for (int x = b * kChunks + t; x < kT * kChunks; x += 128) {
        const int r = x / kChunks;
        uint4* at = reinterpret_cast<uint4*>(v + tile_at(r, x % kChunks));
        if (r >= have) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint32_t* y = reinterpret_cast<uint32_t*>(at);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t z = y[k];
            const bool lo = (z & 0x7f80u) == 0x7f80u, hi = (z & 0x7f800000u) == 0x7f800000u;
            if (lo || hi) {
                y[k] = z & (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
                atomicOr(bad + ((node0 + r) >> 5), 1u << ((node0 + r) & 31));
            }
        }
    }
}
// What the marked nodes that `node` sees add to channel c: the sum of their
// values that are not finite (8-bit: of a row whose scales are not; NaN where
// that is the key's).
template <int TYPE, int D>
__device__ __forceinline__ float not_finite_seen(const TreeParams& p, const TreePiece& w, int node, const uint32_t* bad, int c) {
    float sum = 0.f;
    for (int q = 0; q < 8; ++q) {
        if (!bad[q]) continue;
        for (uint32_t see = bad[q] & mask_word(p, w.e, node, q); see; see &= see - 1) {
            const long long row = tree_row(p.at, w.e, w.h, w.prefix + 32 * q + __ffs(see) - 1);
            if constexpr (TYPE == kTreeE4M3) {
                uint32_t h;  // two halves; the lower one is the code's value
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)static_cast<const uint8_t*>(p.v)[row * D + c]));
                sum += __half2float(__ushort_as_half((uint16_t)h)) * p.v_scale[row];
                if (!isfinite(p.k_scale[row] * p.qscale)) sum = NAN;
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

// One warp brings the token tiles of the CTA's pieces into slots, in ring order,
// by tensor copies of boxes of 128 bytes (64 channels; 8-bit: all, 64 of them
// filled up with zeros, which keeps every row on the 128-byte boundary that a
// copy needs) and 128 rows, or as many rows as a page has: a lane a page. Rows
// past the sequence are whatever the cache (or, where a page is not needed, the
// slot) holds.
template <int TYPE, int D, int NS, typename Order>
__device__ __forceinline__ void copy_tiles(const TreeParams& p, const CUtensorMap* mk, const CUtensorMap* mv,
                                           uint8_t* slots, uint64_t* full, uint64_t* empty, const Waiter& wait,
                                           TreeCursor cur, long long u, long long end) {
    constexpr bool kQ8 = TYPE == kTreeE4M3;
    constexpr int kBlocks = kQ8 ? 1 : D / 64, kSlot = kT * 128 * kBlocks;  // boxes of a row; bytes
    const int lane = lane_id();
    const bool paged = p.at.block_table != nullptr;
    const int shift = p.at.page_shift < 7 ? p.at.page_shift : 7;  // rows of a box, where paged
    Ring<NS> ring;
    unsigned issued = 0;
    TreePiece w;
    while (next_piece(p, cur, u, end, w)) {
        if (w.nodes * p.G - w.mt * p.tile_rows <= 0) continue;
        const int n = w.t1 - w.t0, tokens = w.prefix + w.nodes;
        // the row of this lane's box in a tile (its first one; small pages have more boxes than lanes)
        auto row_of = [&](int tok) {
            int blk = __ldg(p.at.block_table + (size_t)w.e * p.at.max_blocks + (tok >> p.at.page_shift));
            blk = min(max(blk, 0), p.at.num_blocks - 1);
            return (int)((((long long)blk * p.at.hkv + w.h) << p.at.page_shift) + (tok & ((1 << p.at.page_shift) - 1)));
        };
        auto first_row = [&](int k) {
            const int tok = (w.t0 + Order::use(k, n).i) * kT + (lane << shift);
            return tok < tokens && (lane << shift) < kT ? row_of(tok) : 0;
        };
        int row = paged ? first_row(0) : 0;
        for (int k = 0; k < 2 * n; ++k) {
            const RingUse use = Order::use(k, n);
            const int tok0 = (w.t0 + use.i) * kT;
            if (!__all_sync(0xffffffffu, wait(empty + ring.i, ring.ph ^ 1))) {
                // copies in flight land before the block leaves
                for (unsigned x = 1; x <= NS && x <= issued; ++x) {
                    const unsigned j = issued - x;
                    mbar_wait_bounded(full + j % NS, j / NS & 1, p.err, 3, 10000000ull);
                }
                return;
            }
            ++issued;
            const CUtensorMap* map = use.is_v ? mv : mk;
            const uint32_t dst = smem_u32(slots + ring.i * kSlot), bar = smem_u32(full + ring.i);
            auto box = [&](int r, int y) {  // rows from y on to tile rows from r on
#pragma unroll
                for (int c = 0; c < kBlocks; ++c)
                    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                                 "[%0], [%1, {%2, %3}], [%4];"
                                 ::"r"(dst + c * (kT * 128) + r * 128), "l"(map), "r"(c * 64), "r"(y), "r"(bar)
                                 : "memory");
            };
            if (!paged) {
                if (elected()) {
                    mbar_arrive_expect_tx(full + ring.i, kSlot);
                    box(0, (int)(((long long)w.e * p.at.hkv + w.h) * p.at.s_cap) + tok0);
                }
            } else {
                const int have = min(tokens - tok0, kT), boxes = (have + (1 << shift) - 1) >> shift;
                if (elected()) mbar_arrive_expect_tx(full + ring.i, (boxes << shift) * 128 * kBlocks);
                __syncwarp();
                for (int b = lane; b < boxes; b += 32) box(b << shift, b < 32 ? row : row_of(tok0 + (b << shift)));
                if (k + 1 < 2 * n) row = first_row(k + 1);
            }
            ring.next();
        }
    }
}

// Eight warps widen the 8-bit tiles of NR slots into the ring's NS stages: four
// of them every other tile, so that one tile's waits lie under the other's work.
// NR is even: a slot then always is the same four's, which have seen its use
// before (the parity they wait for would also be that of two uses before), and
// copies may land out of order.
template <int D, int NR, int NS>
__device__ __forceinline__ void widen_tiles(const TreeParams& p, const uint8_t* slots, uint64_t* slot_full,
                                            uint64_t* slot_empty, uint8_t* stages, uint64_t* full, uint64_t* empty,
                                            const Waiter& wait, TreeCursor cur, long long u, long long end, int tid) {
    static_assert(NR % 2 == 0 && NS >= 2, "slots of one group");
    constexpr int kC8 = D / 16, kMine = kT * kC8 / 128, kStep = 128 / kC8;  // 16-code chunks of a row, of a thread
    // (the second half of a 128-channel row is another lane's of the next row:
    // eight lanes then store to different banks)
    const unsigned group = tid >> 7;
    const int c = tid % kC8, r0 = ((tid & 127) / kC8) ^ (D == 128 ? c >> 2 : 0);
    const int at0 = tile_at(r0, 2 * c), at1 = tile_at(r0, 2 * c + 1);
    unsigned use = 0;  // of the ring, over all pieces
    TreePiece w;
    while (next_piece(p, cur, u, end, w)) {
        if (w.nodes * p.G - w.mt * p.tile_rows <= 0) continue;
        for (int k = 2 * (w.t1 - w.t0); k > 0; --k, ++use) {
            if ((use & 1) != group) continue;
            const unsigned slot = use % NR, stage = use % NS;
            if (!__all_sync(0xffffffffu, wait(slot_full + slot, use / NR & 1))) return;
            const uint8_t* src = slots + slot * (kT * 128) + r0 * 128 + c * 16;
            uint8_t* dst = stages + stage * (kT * D * 2);
            bool stage_free = false;
#pragma unroll
            for (int h = 0; h < kMine; h += 4) {  // (kStep is a multiple of 8: the rows' places differ by whole groups)
                uint4 x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) x[y] = *reinterpret_cast<const uint4*>(src + (h + y) * kStep * 128);
                if (!stage_free) {
                    if (!__all_sync(0xffffffffu, wait(empty + stage, (use / NS & 1) ^ 1))) return;
                    stage_free = true;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint2 a = widen4(x[y].x), b = widen4(x[y].y), d = widen4(x[y].z), f = widen4(x[y].w);
                    *reinterpret_cast<uint4*>(dst + at0 + (h + y) * kStep * 128) = make_uint4(a.x, a.y, b.x, b.y);
                    *reinterpret_cast<uint4*>(dst + at1 + (h + y) * kStep * 128) = make_uint4(d.x, d.y, f.x, f.y);
                }
            }
            warp_arrive(slot_empty + slot);
            proxy_fence();
            warp_arrive(full + stage);
        }
    }
}

// 64 threads bring a piece's queries: QR rows in blocks of at most 128, zeros
// past its own; 8-bit: channels in the order of widened rows.
template <int D, int QR, bool Q8>
__device__ __forceinline__ void copy_queries(const TreeParams& p, uint8_t* q, uint64_t* q_full, uint64_t* q_empty,
                                             const Waiter& wait, TreeCursor cur, long long u, long long end, int tid) {
    constexpr int kChunks = D / 8, kB = QR < kT ? QR : kT;
    uint32_t ph = 1;  // the first wait passes
    TreePiece w;
    while (next_piece(p, cur, u, end, w)) {
        const int row0 = w.mt * p.tile_rows, rows = w.nodes * p.G - row0;
        if (rows <= 0) continue;
        if (!__all_sync(0xffffffffu, wait(q_empty, ph, kPieceWait))) return;
        ph ^= 1;
        // All of a thread's reads are in flight together: through registers, eight at a
        // time, a piece of 256 rows began with eight waits (64 nodes x 4 heads over 128K
        // 209 us instead of 176, 16 nodes over 4 x 32K 114 instead of 107).
#pragma unroll 4
        for (int x = tid; x < QR * kChunks; x += 64) {
            const int row = x / kChunks, c = x % kChunks;
            const size_t at = row < rows ? q_offset(p, w.e, w.h, row0 + row, D) : 0;
            cp_async16_zfill(q + (row / kB) * kB * D * 2 + tile_at(row % kB, c, kB), static_cast<const uint16_t*>(p.q) + at + c * 8,
                             row < rows);
        }
        cp_async_commit();
        cp_async_wait<0>();
        if constexpr (Q8) {
#pragma unroll 4
            for (int x = tid; x < QR * kChunks; x += 64) {  // (this thread's own)
                const int row = x / kChunks, c = x % kChunks;
                uint4* at = reinterpret_cast<uint4*>(q + (row / kB) * kB * D * 2 + tile_at(row % kB, c, kB));
                const uint4 y = *at;
                *at = make_uint4(__byte_perm(y.x, y.y, 0x5410), __byte_perm(y.x, y.y, 0x7632),
                                 __byte_perm(y.z, y.w, 0x5410), __byte_perm(y.z, y.w, 0x7632));
            }
        }
        proxy_fence();
        warp_arrive(q_full);
    }
}

}  // namespace

// Tensor maps of the caches for copy_tiles (ds_tree_tc.cu).
struct TreeMaps { CUtensorMap k, v; };
cudaError_t make_tree_maps(const TreeParams& p, int type, int d, TreeMaps* m);

}  // namespace ds
