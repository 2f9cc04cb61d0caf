// ds_tree_combine.cu -- joins the pieces of split items of the tree attention.
//
// Row r of an item split into pieces f has maxima m_f, sums l_f and weighted
// values o_f (weights relative to 2^m_f): out = sum_f 2^(m_f - m) o_f /
// sum_f 2^(m_f - m) l_f with m = max m_f. What costs here is latency (a chain
// of a few reads behind the attention's end), so a warp reads the statistics
// of up to 32 pieces at once, a lane a piece, and then keeps eight pieces'
// values in flight. Many pieces (few items): eight warps share a row. Blocks
// belong to items, or, where there are more items than CTAs, to the boundaries
// between the CTAs' shares (a boundary inside an item that has none before).
// The order of the sums is fixed, so results repeat. A block whose every piece
// looked up the split by 64-bit divisions and a walk over the CTAs took 18 to
// 52 us a call; by items and with one division it takes 6 (cold), 20 where 20.6 MB
// of pieces are read (155 pieces of 256 rows: 64 nodes x 4 heads).
#include <math.h>

#include "ds_tree.cuh"

namespace ds {

namespace {

constexpr int kWarps = 8;

template <int D, int WPR>  // WPR warps share a row
__global__ void __launch_bounds__(kWarps * 32) ds_tree_combine_kernel(const __grid_constant__ TreeParams p, int by_item) {
    constexpr int V = D / 32;  // channels of a lane
    __shared__ float sm_o[WPR > 1 ? WPR : 1][D], sm_m[WPR], sm_l[WPR];
    const int warp = warp_id(), lane = lane_id();
    const TreeShares shares(tree_total(p), p.grid);
    const int per = p.hkv * p.n_mt;
    int e = 0, item = 0;
    long long first = 0;
    bool mine = true;
    if (by_item) {
        e = (int)blockIdx.x / per;
        item = (int)blockIdx.x - e * per;
        first = tree_before(p, e) + (long long)item * item_units(p, e);
    } else {
        const long long cut = shares.begin(blockIdx.x + 1);
        mine = cut < shares.begin(p.grid);
        if (mine) {
            const TreeCursor c = tree_seek(p, cut);
            e = c.e;
            item = (int)TreeShares::quotient(cut - c.base, c.units);
            first = c.base + (long long)item * c.units;
            mine = first != cut && first >= shares.begin(blockIdx.x);
        }
    }
    const int units = mine ? item_units(p, e) : 0;
    int i = 0, end = 0;  // CTAs [i, end) have pieces
    if (units > 1) {
        i = shares.holder(first);
        end = shares.holder(first + units - 1) + 1;
    }
    const int h = item / p.n_mt, mt = item - h * p.n_mt;
    const int rows = min(p.tile_rows, tree_nodes(p, e) * p.G - mt * p.tile_rows);  // rows of this tile that exist
    const int r = blockIdx.y * (kWarps / WPR) + warp / WPR, part_warp = warp % WPR;

    // The attention kernel may still be running: its results are complete here.
    // Every block waits, so this launch does not end before that one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (end - i < 2 || r >= rows) return;  // with WPR > 1 the whole block
    // this warp's pieces
    const int n = (end - i + WPR - 1) / WPR, f0 = i + part_warp * n, f1 = min(f0 + n, end);
    float m = -INFINITY, l = 0.f, o[V] = {};
    for (int f = f0; f < f1; f += 32) {
        float mf = -INFINITY, lf = 0.f;
        if (f + lane < f1) {
            const float* part = part_of(p, f + lane, f + lane == i, D);
            mf = part[r];
            lf = part[p.part_rows + r];
        }
        const float mn = fmaxf(m, warp_max(mf)), base = mn == -INFINITY ? 0.f : mn;
        const float old = exp2f(m - base), wf = exp2f(mf - base);
        m = mn;
        l = l * old + warp_sum(lf * wf);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= old;
        const int cnt = min(32, f1 - f);
        for (int g = 0; g < cnt; g += 8) {
            float x[8][V];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = min(g + k, cnt - 1);
                const float* po = part_of(p, f + at, f + at == i, D) + 2 * p.part_rows + (size_t)r * D + lane * V;
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(po);
                    x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(po);
                    x[k][0] = y.x; x[k][1] = y.y;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, wf, g + k);
                if (g + k < cnt) {
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = fmaf(x[k][v], wk, o[v]);
                }
            }
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) { sm_m[warp] = m; sm_l[warp] = l; }
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[warp][lane * V + v] = o[v];
        __syncthreads();
        if (warp > 0) return;
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < WPR; ++k) mx = fmaxf(mx, sm_m[k]);
        if (mx == -INFINITY) mx = 0.f;
        l = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.f;
#pragma unroll
        for (int k = 0; k < WPR; ++k) {
            const float wk = exp2f(sm_m[k] - mx);
            l = fmaf(sm_l[k], wk, l);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = fmaf(sm_o[k][lane * V + v], wk, o[v]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t at = q_offset(p, e, h, mt * p.tile_rows + r, D) + lane * V;
    if (p.out_bf16) {
        uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
        for (int v = 0; v < V; v += 2) out[v / 2] = pack_bf16x2(o[v] * inv, o[v + 1] * inv);
    } else {
        float* out = static_cast<float*>(p.out) + at;
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = o[v] * inv;
    }
}

}  // namespace

cudaError_t launch_tree_combine(const TreeParams& p, int d, cudaStream_t st) {
    if (p.grid < 2) return cudaSuccess;
    const long long items = (long long)p.b * p.hkv * p.n_mt;
    const int by_item = items < p.grid;
    // about grid / items pieces an item: from 16 on, eight warps share a row
    const bool many = p.grid >= 16 * items;
    const int rows = many ? 1 : kWarps;  // of a block
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(by_item ? items : p.grid - 1), (unsigned)((p.part_rows + rows - 1) / rows));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    // launched while the attention kernel still runs; it waits on the device
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (d == 64)
        return many ? cudaLaunchKernelEx(&cfg, ds_tree_combine_kernel<64, kWarps>, p, by_item)
                    : cudaLaunchKernelEx(&cfg, ds_tree_combine_kernel<64, 1>, p, by_item);
    return many ? cudaLaunchKernelEx(&cfg, ds_tree_combine_kernel<128, kWarps>, p, by_item)
                : cudaLaunchKernelEx(&cfg, ds_tree_combine_kernel<128, 1>, p, by_item);
}

}  // namespace ds
