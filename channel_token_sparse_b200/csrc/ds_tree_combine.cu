// ds_tree_combine.cu -- joins the pieces of split items of the tree attention.
//
// Row r of an item split into pieces f has maxima m_f, sums l_f and weighted
// values o_f (weights relative to 2^m_f): out = sum_f 2^(m_f - m) o_f /
// sum_f 2^(m_f - m) l_f with m = max m_f. A block takes eight rows of the item
// that the boundary between two CTAs' shares splits; its warps take pieces in
// turn and are joined in shared memory. An item split over several boundaries
// belongs to the first one. The order of the sums is fixed, so results repeat.
#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kRows = 8;    // rows a block
constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) ds_tree_combine_kernel(const TreeParams p) {
    __shared__ float sm_o[kWarps][kRows][D];
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    // the attention kernel may still be running: its results are complete here
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.x, r0 = blockIdx.y * kRows;
    const long long total = tree_total(p);
    const long long cut = share_begin(total, i + 1, p.grid), mine = share_begin(total, i, p.grid);
    if (cut == mine || cut >= total) return;
    TreeCursor c = tree_seek(p, cut);
    const int per = p.hkv * p.n_mt;
    if (cut == c.base) return;  // the boundary is an entry's
    const int item = (int)((cut - c.base) / c.units);
    const long long first = c.base + (long long)item * c.units, last = first + c.units;
    if (first == cut || first < mine) return;  // an item's boundary, or an earlier one's item
    (void)per;
    TreePiece w;
    w.e = c.e; w.h = item / p.n_mt; w.mt = item - w.h * p.n_mt;
    w.prefix = c.prefix; w.nodes = c.nodes;
    const int rows = min(p.tile_rows, w.nodes * p.G - w.mt * p.tile_rows);  // rows of this tile that exist
    if (r0 >= rows) return;
    const int nr = min(kRows, rows - r0);
    int end = i + 1;  // CTAs [i, end) hold units of the item
    while (end < p.grid && share_begin(total, end, p.grid) < last) ++end;

    const int warp = warp_id(), lane = lane_id();
    constexpr int V = D / 32;  // channels of a lane
    float m[kRows], l[kRows], o[kRows][V];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[r][v] = 0.f;
    }
    for (int f = i + warp; f < end; f += kWarps) {
        if (share_begin(total, f, p.grid) == share_begin(total, f + 1, p.grid)) continue;  // an empty share
        const float* part = part_of(p, f, f == i, D);
        const float* po = part + 2 * p.part_rows + (size_t)r0 * D;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r < nr) {
                const float mf = part[r0 + r], lf = part[p.part_rows + r0 + r];
                const float mn = fmaxf(m[r], mf);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float wa = exp2f(m[r] - base), wb = exp2f(mf - base);
                m[r] = mn;
                l[r] = l[r] * wa + lf * wb;
#pragma unroll
                for (int v = 0; v < V; ++v) o[r][v] = o[r][v] * wa + po[(size_t)r * D + v * 32 + lane] * wb;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (lane == 0) { sm_m[warp][r] = m[r]; sm_l[warp][r] = l[r]; }
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[warp][r][v * 32 + lane] = o[r][v];
    }
    __syncthreads();
    const int r = warp;
    if (r >= nr) return;
    float mx = -INFINITY;
#pragma unroll
    for (int f = 0; f < kWarps; ++f) mx = fmaxf(mx, sm_m[f][r]);
    if (mx == -INFINITY) mx = 0.f;
    float sum = 0.f, acc[V] = {};
#pragma unroll
    for (int f = 0; f < kWarps; ++f) {
        const float wf = exp2f(sm_m[f][r] - mx);
        sum += sm_l[f][r] * wf;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += sm_o[f][r][v * 32 + lane] * wf;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t at = q_offset(p, w.e, w.h, w.mt * p.tile_rows + r0 + r, D);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float x = acc[v] * inv;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at + v * 32 + lane] = __float2bfloat16_rn(x);
        else static_cast<float*>(p.out)[at + v * 32 + lane] = x;
    }
}

}  // namespace

cudaError_t launch_tree_combine(const TreeParams& p, int d, cudaStream_t st) {
    if (p.grid < 2) return cudaSuccess;
    // launched while the attention kernel still runs; it waits on the device
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.grid - 1), (unsigned)((p.part_rows + kRows - 1) / kRows));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return d == 64 ? cudaLaunchKernelEx(&cfg, ds_tree_combine_kernel<64>, p)
                   : cudaLaunchKernelEx(&cfg, ds_tree_combine_kernel<128>, p);
}

}  // namespace ds
