// ds_tree_api.cu -- C ABI of the cache writes and reads and of the tree
// attention: argument validation and dispatch. Contract: include/ds.h.
#include <math.h>

#include "ds.h"
#include "ds_internal.h"
#include "ds_tree.cuh"

namespace {

using ds::CacheRows;

#define DS_FAIL(...) return static_cast<ds_status>(ds::report(__VA_ARGS__))

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Every pointer of the list is NULL or aligned.
template <typename... P> bool all_aligned(size_t n, P... p) { return (aligned(p, n) && ...); }

ds_status launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return DS_OK;
    DS_FAIL(DS_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Whether a * b * c rows (a, b >= 1) of d channels reach 2^40 elements. The
// products of two sizes fit 64 bits, those of three do not.
bool too_large(long long a, long long b, long long c, int d) {
    const long long most = ((1ll << 40) - 1) / d;
    return a * b > most || c > most / (a * b);
}

struct Pool {
    const int32_t* table = nullptr;
    int max_blocks = 0, page_size = 0, num_blocks = 0;
};

// Fills `at` (and the rows an entry can address) for a dense or paged cache.
ds_status cache_rows(const Pool* pool, int b, int hkv, int s_cap, int d, CacheRows* at, int* rows) {
    at->hkv = hkv;
    if (!pool) {
        if (s_cap < 1) DS_FAIL(DS_ERR_INVALID_ARG, "s_cap (%d) must be >= 1", s_cap);
        if (too_large(b, hkv, s_cap, d)) DS_FAIL(DS_ERR_UNSUPPORTED, "cache too large");
        at->s_cap = s_cap;
        *rows = s_cap;
        return DS_OK;
    }
    if (!pool->table) DS_FAIL(DS_ERR_INVALID_ARG, "block_table is NULL");
    if (!aligned(pool->table, 4)) DS_FAIL(DS_ERR_INVALID_ARG, "block_table not 4-byte aligned");
    int shift = 0;
    while (shift < 16 && (1 << shift) < pool->page_size) ++shift;
    if (pool->page_size < 1 || (1 << shift) != pool->page_size)
        DS_FAIL(DS_ERR_INVALID_ARG, "page_size %d must be a power of two in [1, 65536]", pool->page_size);
    if (pool->num_blocks < 1 || pool->max_blocks < 1)
        DS_FAIL(DS_ERR_INVALID_ARG, "num_blocks and max_blocks must be >= 1");
    if (too_large(pool->num_blocks, hkv, 1 << shift, d)) DS_FAIL(DS_ERR_UNSUPPORTED, "pool too large");
    const long long r = (long long)pool->max_blocks << shift;
    at->block_table = pool->table;
    at->max_blocks = pool->max_blocks;
    at->page_shift = shift;
    at->num_blocks = pool->num_blocks;
    *rows = r > 0x7fffffff ? 0x7fffffff : (int)r;
    return DS_OK;
}

ds_status check_heads(int b, int hq, int hkv, int d) {
    if (b < 1 || hq < 1 || hkv < 1) DS_FAIL(DS_ERR_INVALID_ARG, "b, hq and hkv must be >= 1");
    if (d != 64 && d != 128) DS_FAIL(DS_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", d);
    return DS_OK;
}

ds_status write_kv(const void* q, long long q_bs, long long q_ts, const void* k, long long k_bs, long long k_ts,
                   const void* v, long long v_bs, long long v_ts, ds_dtype dt, const void* q_weight,
                   const void* k_weight, float eps, const float* inv_freq, int rot_dim, ds_rope rope,
                   const int32_t* positions, const int32_t* starts, const int32_t* lens, int b, int t, int hq,
                   int hkv, int s_cap, int d, void* q_out, void* k_cache, void* v_cache, ds_dtype cache_dt,
                   float* k_scale, float* v_scale, const Pool* pool, cudaStream_t stream) {
    ds_status r = check_heads(b, q ? hq : 1, hkv, d);
    if (r != DS_OK) return r;
    if (t < 1) DS_FAIL(DS_ERR_INVALID_ARG, "t (%d) must be >= 1", t);
    if ((long long)b * t > (1ll << 30)) DS_FAIL(DS_ERR_UNSUPPORTED, "b * t > 2^30");
    if (hkv > (1 << 20) || (q && hq > (1 << 20))) DS_FAIL(DS_ERR_UNSUPPORTED, "too many heads");
    if (dt != DS_F32 && dt != DS_BF16) DS_FAIL(DS_ERR_UNSUPPORTED, "dtype %d (supported: f32, bf16)", (int)dt);
    if (cache_dt != dt && cache_dt != DS_E4M3)
        DS_FAIL(DS_ERR_UNSUPPORTED, "cache dtype %d (supported: that of q/k/v, e4m3)", (int)cache_dt);
    if (!k || !v || !k_cache || !v_cache) DS_FAIL(DS_ERR_INVALID_ARG, "k, v, k_cache or v_cache is NULL");
    if ((q == nullptr) != (q_out == nullptr)) DS_FAIL(DS_ERR_INVALID_ARG, "give both q and q_out or neither");
    if (cache_dt == DS_E4M3 && (!k_scale || !v_scale))
        DS_FAIL(DS_ERR_INVALID_ARG, "an 8-bit cache needs k_scale and v_scale");
    if ((q_weight || k_weight) && !(eps >= 0.f)) DS_FAIL(DS_ERR_INVALID_ARG, "eps must be >= 0");
    if (inv_freq) {
        if (rot_dim < 16 || rot_dim > d || rot_dim % 16)
            DS_FAIL(DS_ERR_INVALID_ARG, "rot_dim %d must be a multiple of 16 in [16, d]", rot_dim);
        if (rope != DS_ROPE_HALF && rope != DS_ROPE_INTERLEAVED)
            DS_FAIL(DS_ERR_INVALID_ARG, "unknown rotation style %d", (int)rope);
    }
    if (!all_aligned(16, q, k, v, q_weight, k_weight, (const void*)q_out, (const void*)k_cache, (const void*)v_cache))
        DS_FAIL(DS_ERR_INVALID_ARG, "pointer not 16-byte aligned");
    if (!all_aligned(4, inv_freq, positions, starts, lens, (const float*)k_scale, (const float*)v_scale))
        DS_FAIL(DS_ERR_INVALID_ARG, "pointer not 4-byte aligned");
    const int unit = dt == DS_F32 ? 4 : 8;  // elements of 16 bytes
    for (long long x : {q ? q_bs : 0ll, q ? q_ts : 0ll, k_bs, k_ts, v_bs, v_ts})
        if (x % unit) DS_FAIL(DS_ERR_INVALID_ARG, "stride %lld is not a multiple of 16 bytes", x);
    ds::WriteArgs a{};
    if ((r = cache_rows(pool, b, hkv, s_cap, d, &a.at, &a.rows)) != DS_OK) return r;
    a.q = q; a.k = k; a.v = v;
    a.q_bs = q_bs; a.q_ts = q_ts; a.k_bs = k_bs; a.k_ts = k_ts; a.v_bs = v_bs; a.v_ts = v_ts;
    a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps;
    a.inv_freq = inv_freq; a.rot_dim = rot_dim; a.interleaved = rope == DS_ROPE_INTERLEAVED;
    a.positions = positions; a.starts = starts; a.lens = lens;
    a.b = b; a.t = t; a.hq = hq; a.hkv = hkv; a.d = d;
    a.f32 = dt == DS_F32; a.e4m3 = cache_dt == DS_E4M3;
    a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    return launched(ds::launch_write_kv(a, stream), "cache write launch");
}

ds_status read_kv(const void* k, const void* v, const float* k_scale, const float* v_scale, const int32_t* seq_lens,
                  int b, int hkv, int s, int s_cap, int d, void* k_out, void* v_out, ds_dtype out_dt, int s_out_cap,
                  const Pool* pool, cudaStream_t stream) {
    ds_status r = check_heads(b, hkv, hkv, d);
    if (r != DS_OK) return r;
    if (out_dt != DS_F32 && out_dt != DS_BF16)
        DS_FAIL(DS_ERR_UNSUPPORTED, "out dtype %d (supported: f32, bf16)", (int)out_dt);
    // an empty output (s = 0) may have no address
    if (!k || !k_scale || (!k_out && s != 0)) DS_FAIL(DS_ERR_INVALID_ARG, "k_cache, k_scale or k_out is NULL");
    if (((v == nullptr) != (v_out == nullptr) && s != 0) || (v == nullptr) != (v_scale == nullptr))
        DS_FAIL(DS_ERR_INVALID_ARG, "give all of v_cache, v_scale and v_out or none");
    if (!all_aligned(16, k, v, (const void*)k_out, (const void*)v_out))
        DS_FAIL(DS_ERR_INVALID_ARG, "pointer not 16-byte aligned");
    if (!all_aligned(4, k_scale, v_scale, seq_lens)) DS_FAIL(DS_ERR_INVALID_ARG, "pointer not 4-byte aligned");
    ds::ReadArgs a{};
    int rows = 0;
    if ((r = cache_rows(pool, b, hkv, s_cap, d, &a.at, &rows)) != DS_OK) return r;
    if (s < 0 || s > rows || s > s_out_cap)
        DS_FAIL(DS_ERR_INVALID_ARG, "need 0 <= s (%d) <= cache rows (%d) and s_out_cap (%d)", s, rows, s_out_cap);
    if (too_large(b, hkv, s_out_cap, d)) DS_FAIL(DS_ERR_UNSUPPORTED, "output too large");
    if (s == 0) return DS_OK;
    a.k = k; a.v = v; a.k_scale = k_scale; a.v_scale = v_scale; a.seq_lens = seq_lens;
    a.b = b; a.hkv = hkv; a.s = s; a.d = d; a.k_out = k_out; a.v_out = v_out;
    a.f32 = out_dt == DS_F32; a.s_out_cap = s_out_cap;
    return launched(ds::launch_read_kv(a, stream), "cache read launch");
}

struct TreeShape { int type; ds::TreePlan plan; int grid, n_mt, part_rows; size_t parts, ws; };

ds_status tree_shape(int b, int t, int hq, int hkv, int s, int d, ds_dtype kvdt, TreeShape* o) {
    ds_status r = check_heads(b, hq, hkv, d);
    if (r != DS_OK) return r;
    if (hq % hkv) DS_FAIL(DS_ERR_INVALID_ARG, "hq (%d) must be a multiple of hkv (%d)", hq, hkv);
    if (hq / hkv > 8) DS_FAIL(DS_ERR_UNSUPPORTED, "hq/hkv = %d > 8", hq / hkv);
    if (t < 1) DS_FAIL(DS_ERR_INVALID_ARG, "t (%d) must be >= 1", t);
    if (t > 256) DS_FAIL(DS_ERR_UNSUPPORTED, "t = %d > 256 drafted tokens", t);
    if (s < 0) DS_FAIL(DS_ERR_INVALID_ARG, "s (%d) must be >= 0", s);
    if (s > 0x7fffffff - 1024) DS_FAIL(DS_ERR_UNSUPPORTED, "s = %d too large", s);
    if ((long long)b * hkv > (1ll << 26)) DS_FAIL(DS_ERR_UNSUPPORTED, "too many rows");
    if (kvdt != DS_F32 && kvdt != DS_BF16 && kvdt != DS_E4M3)
        DS_FAIL(DS_ERR_UNSUPPORTED, "k/v dtype %d (supported: f32, bf16, e4m3)", (int)kvdt);
    o->type = kvdt == DS_F32 ? ds::kTreeF32 : kvdt == DS_BF16 ? ds::kTreeBF16 : ds::kTreeE4M3;
    const int rows = t * (hq / hkv);
    o->plan = o->type == ds::kTreeF32 ? ds::plan_tree_simt(rows, d) : ds::plan_tree_tc(rows, o->type);
    o->n_mt = (rows + o->plan.tile_rows - 1) / o->plan.tile_rows;
    // a multiple of 4 keeps every place, and the values behind its rows' statistics, 16-byte aligned
    o->part_rows = ((rows < o->plan.tile_rows ? rows : o->plan.tile_rows) + 3) / 4 * 4;
    const long long tiles = ((long long)s + t + o->plan.tile_tokens - 1) / o->plan.tile_tokens;
    const long long units = (long long)b * hkv * o->n_mt * tiles;
    o->grid = units < o->plan.grid ? (int)units : o->plan.grid;
    // two places a CTA for pieces of split items
    o->ws = o->parts = (size_t)o->grid * 2 * o->part_rows * (d + 2) * 4;
    if (o->type != ds::kTreeF32) {  // a piece has an item's tiles at most, and a CTA's share of all
        const long long share = (units + o->grid - 1) / o->grid;
        o->ws += ds::tree_tc_sums(o->plan, o->grid, tiles < share ? tiles : share, d);
    }
    return DS_OK;
}

ds_status tree_decode(const void* q, const void* k, const void* v, ds_dtype kvdt, const float* k_scale,
                      const float* v_scale, const int32_t* mask, const int32_t* seq_lens, const int32_t* node_lens,
                      int b, int t, int hq, int hkv, int s, int s_cap, int d, float sm_scale, void* out,
                      ds_dtype out_dt, void* ws, size_t ws_bytes, const Pool* pool, cudaStream_t stream) {
    TreeShape sh;
    ds_status r = tree_shape(b, t, hq, hkv, s, d, kvdt, &sh);
    if (r != DS_OK) return r;
    if (!q || !k || !v || !out) DS_FAIL(DS_ERR_INVALID_ARG, "q, k, v or out is NULL");
    if (kvdt == DS_E4M3 && (!k_scale || !v_scale))
        DS_FAIL(DS_ERR_INVALID_ARG, "an 8-bit cache needs k_scale and v_scale");
    if (!(out_dt == DS_F32 || (out_dt == DS_BF16 && kvdt != DS_F32)))
        DS_FAIL(DS_ERR_INVALID_ARG, "out dtype must be DS_F32 or (with bf16 or 8-bit k/v) DS_BF16");
    if (!(sm_scale == sm_scale)) DS_FAIL(DS_ERR_INVALID_ARG, "sm_scale is NaN");
    if (!all_aligned(16, q, k, v, (const void*)out, (const void*)ws))
        DS_FAIL(DS_ERR_INVALID_ARG, "pointer not 16-byte aligned");
    if (!all_aligned(4, k_scale, v_scale, mask, seq_lens, node_lens))
        DS_FAIL(DS_ERR_INVALID_ARG, "pointer not 4-byte aligned");
    ds::TreeParams p{};
    int rows = 0;
    if ((r = cache_rows(pool, b, hkv, s_cap, d, &p.at, &rows)) != DS_OK) return r;
    if ((long long)s + t > rows)
        DS_FAIL(DS_ERR_INVALID_ARG, "need s (%d) + t (%d) <= cache rows (%d)", s, t, rows);
    if (ws_bytes < sh.ws || !ws) DS_FAIL(DS_ERR_WORKSPACE, "workspace %zu B < required %zu B", ws ? ws_bytes : 0, sh.ws);
    p.q = q; p.k = k; p.v = v; p.k_scale = k_scale; p.v_scale = v_scale;
    p.mask = mask; p.seq_lens = seq_lens; p.node_lens = node_lens;
    p.b = b; p.t = t; p.hq = hq; p.hkv = hkv; p.G = hq / hkv; p.s = s;
    p.rows = t * p.G;
    p.cache_rows = pool ? (long long)pool->num_blocks * hkv << p.at.page_shift : (long long)b * hkv * s_cap;
    if (p.cache_rows > 0x7fffffffll - 256) DS_FAIL(DS_ERR_UNSUPPORTED, "a cache of 2^31 rows");
    p.tile_rows = sh.plan.tile_rows; p.tile_tokens = sh.plan.tile_tokens;
    p.n_mt = sh.n_mt; p.part_rows = sh.part_rows; p.grid = sh.grid;
    p.qscale = (sm_scale > 0.f ? sm_scale : 1.0f / sqrtf((float)d)) * 1.4426950408889634f;
    p.out = out; p.out_bf16 = out_dt == DS_BF16;
    p.part = static_cast<float*>(ws);
    p.sums = sh.ws > sh.parts ? p.part + sh.parts / 4 : nullptr;
    cudaError_t e = ds::device_status_word(&p.err);
    if (e != cudaSuccess) return launched(e, "cudaGetSymbolAddress");
    e = sh.type == ds::kTreeF32 ? ds::launch_tree_simt(p, d, stream) : ds::launch_tree_tc(p, sh.type, d, stream);
    if (e == cudaSuccess) e = ds::launch_tree_combine(p, d, stream);
    return launched(e, "tree decode launch");
}

}  // namespace

extern "C" {

ds_status ds_write_kv(const void* q, long long q_bs, long long q_ts, const void* k, long long k_bs, long long k_ts,
                      const void* v, long long v_bs, long long v_ts, ds_dtype dt, const void* q_weight,
                      const void* k_weight, float eps, const float* inv_freq, int rot_dim, ds_rope rope,
                      const int32_t* positions, const int32_t* starts, const int32_t* lens, int b, int t, int hq,
                      int hkv, int s_cap, int d, void* q_out, void* k_cache, void* v_cache, ds_dtype cache_dt,
                      float* k_scale, float* v_scale, cudaStream_t stream) {
    return write_kv(q, q_bs, q_ts, k, k_bs, k_ts, v, v_bs, v_ts, dt, q_weight, k_weight, eps, inv_freq, rot_dim, rope,
                    positions, starts, lens, b, t, hq, hkv, s_cap, d, q_out, k_cache, v_cache, cache_dt, k_scale,
                    v_scale, nullptr, stream);
}

ds_status ds_write_kv_paged(const void* q, long long q_bs, long long q_ts, const void* k, long long k_bs,
                            long long k_ts, const void* v, long long v_bs, long long v_ts, ds_dtype dt,
                            const void* q_weight, const void* k_weight, float eps, const float* inv_freq, int rot_dim,
                            ds_rope rope, const int32_t* positions, const int32_t* starts, const int32_t* lens, int b,
                            int t, int hq, int hkv, int d, void* q_out, void* k_pool, void* v_pool, ds_dtype cache_dt,
                            float* k_scale, float* v_scale, const int32_t* block_table, int max_blocks, int page_size,
                            int num_blocks, cudaStream_t stream) {
    const Pool pool{block_table, max_blocks, page_size, num_blocks};
    return write_kv(q, q_bs, q_ts, k, k_bs, k_ts, v, v_bs, v_ts, dt, q_weight, k_weight, eps, inv_freq, rot_dim, rope,
                    positions, starts, lens, b, t, hq, hkv, 0, d, q_out, k_pool, v_pool, cache_dt, k_scale, v_scale,
                    &pool, stream);
}

ds_status ds_read_kv(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                     const int32_t* seq_lens, int b, int hkv, int s, int s_cap, int d, void* k_out, void* v_out,
                     ds_dtype out_dt, int s_out_cap, cudaStream_t stream) {
    return read_kv(k_cache, v_cache, k_scale, v_scale, seq_lens, b, hkv, s, s_cap, d, k_out, v_out, out_dt, s_out_cap,
                   nullptr, stream);
}

ds_status ds_read_kv_paged(const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
                           const int32_t* block_table, int max_blocks, int page_size, int num_blocks,
                           const int32_t* seq_lens, int b, int hkv, int s, int d, void* k_out, void* v_out,
                           ds_dtype out_dt, int s_out_cap, cudaStream_t stream) {
    const Pool pool{block_table, max_blocks, page_size, num_blocks};
    return read_kv(k_pool, v_pool, k_scale, v_scale, seq_lens, b, hkv, s, 0, d, k_out, v_out, out_dt, s_out_cap, &pool,
                   stream);
}

ds_status ds_tree_decode_workspace_size(int b, int t, int hq, int hkv, int s, int d, ds_dtype kvdt, size_t* bytes) {
    if (!bytes) DS_FAIL(DS_ERR_INVALID_ARG, "bytes is NULL");
    TreeShape sh;
    ds_status r = tree_shape(b, t, hq, hkv, s, d, kvdt, &sh);
    if (r != DS_OK) return r;
    *bytes = sh.ws;
    return DS_OK;
}

ds_status ds_tree_decode(const void* q, const void* k, const void* v, ds_dtype kvdt, const float* k_scale,
                         const float* v_scale, const int32_t* mask, const int32_t* seq_lens, const int32_t* node_lens,
                         int b, int t, int hq, int hkv, int s, int s_cap, int d, float sm_scale, void* out,
                         ds_dtype out_dt, void* ws, size_t ws_bytes, cudaStream_t stream) {
    return tree_decode(q, k, v, kvdt, k_scale, v_scale, mask, seq_lens, node_lens, b, t, hq, hkv, s, s_cap, d,
                       sm_scale, out, out_dt, ws, ws_bytes, nullptr, stream);
}

ds_status ds_tree_decode_paged(const void* q, const void* k_pool, const void* v_pool, ds_dtype kvdt,
                               const float* k_scale, const float* v_scale, const int32_t* mask,
                               const int32_t* block_table, int max_blocks, int page_size, int num_blocks,
                               const int32_t* seq_lens, const int32_t* node_lens, int b, int t, int hq, int hkv, int s,
                               int d, float sm_scale, void* out, ds_dtype out_dt, void* ws, size_t ws_bytes,
                               cudaStream_t stream) {
    const Pool pool{block_table, max_blocks, page_size, num_blocks};
    return tree_decode(q, k_pool, v_pool, kvdt, k_scale, v_scale, mask, seq_lens, node_lens, b, t, hq, hkv, s, 0, d,
                       sm_scale, out, out_dt, ws, ws_bytes, &pool, stream);
}

}  // extern "C"
