// ds_tree_simt.cu -- tree attention over fp32 caches, on the CUDA cores.
//
// One pass over an item's tokens with the running maximum and sum of each
// row's softmax: for a tile of 64 tokens the scores s = qscale * q.k (base-2
// exponents) of 8 to 32 query rows, their new maxima, weights 2^(s - m), and the
// weighted values, all in fp32. A tile's K and V rows are read into
// shared memory once and serve the row tile. Kept simple: fp32 caches are the
// small and the reference ones (4 nodes over 512 tokens: 11.4 us, two launches'
// latency; 8 nodes x 4 heads over 4 x 4K 166 us against 21 us of bytes: the tile of
// keys is read from shared memory once a row).
#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kNT = 256;
// Query rows of a row tile: 32, or few (a tile costs its rows' arithmetic whether
// they exist or not; four channels a thread at least): see plan_tree_simt.
constexpr int kMany = 32;
template <int D> constexpr int kFew = D == 128 ? 8 : 16;
constexpr int kT = 64;     // tokens of a token tile

template <int D, int kR> constexpr int simt_smem() { return (kR * D + kT * (D + 4) + kT * D + kR * (kT + 4) + 3 * kR) * 4; }

template <int D, int kR>
__global__ void __launch_bounds__(kNT) ds_tree_simt_kernel(const __grid_constant__ TreeParams p) {
    extern __shared__ __align__(16) float sm[];
    float* sq = sm;                     // [kR][D] queries, times qscale
    float* sk = sq + kR * D;            // [kT][D + 4]
    float* sv = sk + kT * (D + 4);      // [kT][D]
    float* ss = sv + kT * D;            // [kR][kT + 4] scores, then weights
    float* s_m = ss + kR * (kT + 4);    // [kR] running maximum
    float* s_l = s_m + kR;              // [kR] running sum
    float* s_w = s_l + kR;              // [kR] factor of what was summed so far
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tid = threadIdx.x;
    const TreeShares shares(tree_total(p), p.grid);
    long long u = shares.begin(blockIdx.x);
    const long long end = shares.begin(blockIdx.x + 1);
    if (u >= end) return;
    TreeCursor cur = tree_seek(p, u);
    TreePiece w;
    constexpr int kC = kNT / kR;        // threads of a row
    constexpr int kO = D / kC;          // output channels of a thread
    const int orow = tid / kC, oc = (tid % kC) * 4;  // its row; channels oc + 4 kC j ..
    while (next_piece(p, cur, u, end, w)) {
        const int row0 = w.mt * p.tile_rows;
        const int rows = min(kR, w.nodes * p.G - row0);
        // row tiles of nodes that do not exist in this entry: nothing to do
        if (rows <= 0) continue;
        __syncthreads();
        for (int x = tid; x < kR * D / 4; x += kNT) {
            const int r = x / (D / 4), c = x % (D / 4) * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const size_t at = q_offset(p, w.e, w.h, row0 + r, D) + c;
                f = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at);
            }
            f.x *= p.qscale; f.y *= p.qscale; f.z *= p.qscale; f.w *= p.qscale;
            *reinterpret_cast<float4*>(sq + r * D + c) = f;
        }
        if (tid < kR) { s_m[tid] = -INFINITY; s_l[tid] = 0.f; }
        float o[kO];
#pragma unroll
        for (int j = 0; j < kO; ++j) o[j] = 0.f;

        for (int tile = w.t0; tile < w.t1; ++tile) {
            const int tok0 = tile * kT;
            const int ntok = min(kT, w.prefix + w.nodes - tok0);
            constexpr int kL = kT * D / 4 / kNT;  // 16-byte pieces of a thread: all read before the first is stored
            float4 fk[kL], fv[kL];
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const int x = tid + j * kNT, t = x / (D / 4), c = x % (D / 4) * 4;
                fk[j] = fv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t < ntok) {
                    const long long row = tree_row(p.at, w.e, w.h, tok0 + t);
                    fk[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.k) + row * D + c);
                    fv[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.v) + row * D + c);
                }
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const int x = tid + j * kNT, t = x / (D / 4), c = x % (D / 4) * 4;
                *reinterpret_cast<float4*>(sk + t * (D + 4) + c) = fk[j];
                *reinterpret_cast<float4*>(sv + t * D + c) = fv[j];
            }
            __syncthreads();
            // scores: a thread takes one row and tokens t = tid % kC + kC j
            {
                const int r = tid / kC;
                float acc[kT / kC] = {};
                for (int c = 0; c < D; c += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(sq + r * D + c);
#pragma unroll
                    for (int j = 0; j < kT / kC; ++j) {
                        const float4 b = *reinterpret_cast<const float4*>(sk + (tid % kC + kC * j) * (D + 4) + c);
                        acc[j] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc[j]))));
                    }
                }
                const int node = (row0 + r) / p.G;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < kT / kC; ++j) {
                    const int t = tid % kC + kC * j, tok = tok0 + t - w.prefix;  // node index of the token
                    bool sees = r < rows && t < ntok;
                    if (sees && tok >= 0) sees = mask_word(p, w.e, node, tok >> 5) >> (tok & 31) & 1;
                    acc[j] = sees ? acc[j] : -INFINITY;
                    mx = fmaxf(mx, acc[j]);
                }
#pragma unroll
                for (int x = 1; x < kC; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float m_old = s_m[r], m_new = fmaxf(m_old, mx);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < kT / kC; ++j) {
                    const float e = exp2f(acc[j] - base);
                    ss[r * (kT + 4) + tid % kC + kC * j] = e;
                    sum += e;
                }
#pragma unroll
                for (int x = 1; x < kC; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                __syncwarp();
                if (tid % kC == 0) {
                    const float f = exp2f(m_old - base);
                    s_w[r] = f;
                    s_l[r] = s_l[r] * f + sum;
                    s_m[r] = m_new;
                }
            }
            __syncthreads();
            {
                const float f = s_w[orow];
#pragma unroll
                for (int j = 0; j < kO; ++j) o[j] *= f;
                auto add = [&](int t, float e) {
#pragma unroll
                    for (int j = 0; j < kO / 4; ++j) {
                        const float4 v = *reinterpret_cast<const float4*>(sv + t * D + oc + 4 * kC * j);
                        o[4 * j + 0] = fmaf(e, v.x, o[4 * j + 0]);
                        o[4 * j + 1] = fmaf(e, v.y, o[4 * j + 1]);
                        o[4 * j + 2] = fmaf(e, v.z, o[4 * j + 2]);
                        o[4 * j + 3] = fmaf(e, v.w, o[4 * j + 3]);
                    }
                };
                const float* e = ss + orow * (kT + 4);
                if (tok0 + kT <= w.prefix) {
#pragma unroll 4
                    for (int t = 0; t < kT; ++t) add(t, e[t]);
                } else {
                    for (int t = 0; t < ntok; ++t)
                        if (e[t] != 0.f) add(t, e[t]);  // a masked token does not count, whatever its values are
                }
            }
        }
        if (orow < rows) {
            const float l = s_l[orow];
            if (w.whole()) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const size_t at = q_offset(p, w.e, w.h, row0 + orow, D);
#pragma unroll
                for (int j = 0; j < kO; ++j) {
                    const size_t x = at + oc + 4 * kC * (j / 4) + j % 4;
                    static_cast<float*>(p.out)[x] = o[j] * inv;
                }
            } else {
                float* part = part_of(p, blockIdx.x, w.t0 == 0, D);
                if (tid % kC == 0) { part[orow] = s_m[orow]; part[p.part_rows + orow] = l; }
                float* po = part + 2 * p.part_rows + (size_t)orow * D;
#pragma unroll
                for (int j = 0; j < kO; ++j) po[oc + 4 * kC * (j / 4) + j % 4] = o[j];
            }
        }
    }
}

template <int D, int R>
cudaError_t run(const TreeParams& p, cudaStream_t st) {
    static_assert(simt_smem<D, R>() <= 227 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(ds_tree_simt_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         simt_smem<D, R>());
    if (e != cudaSuccess) return e;
    ds_tree_simt_kernel<D, R><<<p.grid, kNT, simt_smem<D, R>(), st>>>(p);
    return cudaGetLastError();
}

}  // namespace

TreePlan plan_tree_simt(int rows, int d) {
    // A tile of few rows takes a third (64 channels: five ninths) of the time of one of
    // 32. One or more of them against the others, us a call of 8 kv heads over 2 x 16K:
    //   128 channels  8 rows 108 or 297; 9 to 16 201 or 297; 17 to 24 295 or 299;
    //                 25 to 32 385 or 299; 33 to 40 483 or 585; 41 to 48 578 or 585; 64 756 or 585
    //   64 channels   16 rows 93 or 162; 17 to 32 178 or 162; 33 to 48 258 or 312; 64 344 or 312
    const int few = d == 64 ? kFew<64> : kFew<128>;
    const int n_few = (rows + few - 1) / few, n_many = (rows + kMany - 1) / kMany;
    const bool cheaper = d == 64 ? 5 * n_few <= 9 * n_many : n_few <= 3 * n_many;
    return TreePlan{cheaper ? few : kMany, kT, 2 * 148};
}

cudaError_t launch_tree_simt(const TreeParams& p, int d, cudaStream_t st) {
    if (p.tile_rows == kMany) return d == 64 ? run<64, kMany>(p, st) : run<128, kMany>(p, st);
    return d == 64 ? run<64, kFew<64>>(p, st) : run<128, kFew<128>>(p, st);
}

}  // namespace ds
