// ds_kv.cu -- writing new tokens' rows into K/V caches (per-head norm, position
// rotation and 8-bit quantisation in the storing pass) and reading 8-bit rows
// back, for sm_100a.
//
// Write: a head's vector x [d] becomes y = x * w * rsqrt(mean(x^2) + eps), the
// pairs of its first rot channels turn by position * inv_freq, and y is stored
// in the destination's type; an 8-bit row stores scale = max(amax / 448,
// 2^-126) and code = e4m3_rn(y / scale). Each value is read once and written
// once, so bandwidth bounds it. d / 16 lanes own a head's vector (16 channels
// each, as two 8-channel chunks that hold whole rotation pairs), so the norm
// and the amax are short butterflies and no value leaves its lane. A warp
// keeps one token: its angles (64-bit product and reduction, then one fp32
// sine and cosine each) are computed once and serve all of its heads.
//
// Measured on a B200: 8192 tokens of 32 + 8 + 8 heads of 128 in bf16, 201 MB,
// 47.5 us (65 % of the copy rate: the chain from a head's load to its store), in
// fp32 70 us (87 %); into 8-bit pages 51 us (the same chain, and issue); 32 single
// tokens 6 us in the kernel.
//
// Read: 16 codes a thread and step, times the row's scale. 65536 rows of 8
// heads, 407 MB: 71 us, 87 % of the copy rate.
#include "ds_common.cuh"
#include "ds_internal.h"

namespace ds {

namespace {

constexpr int kKvNT = 256;

// e4m3 codes of two values (lo in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 codes -> fp32 values (exact: e4m3 is a subset of fp16).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// x / s correctly rounded, from r = 1 / s correctly rounded (Markstein 1990:
// one residual corrects the product), for quotients that do not underflow; a
// division instruction sequence each was what bounded 8-bit writes.
__device__ __forceinline__ float divide(float x, float s, float r) {
    const float q = __fmul_rn(x, r);
    return fmaf(fmaf(-q, s, x), r, q);
}
// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight consecutive channels.
template <typename T> __device__ __forceinline__ void load8(float (&x)[8], const T* p);
template <> __device__ __forceinline__ void load8<float>(float (&x)[8], const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], c = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = c.x; x[5] = c.y; x[6] = c.z; x[7] = c.w;
}
template <> __device__ __forceinline__ void load8<bf16_t>(float (&x)[8], const bf16_t* p) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&x)[8]) {
    uint4 w;
    w.x = pack_bf16x2(x[0], x[1]); w.y = pack_bf16x2(x[2], x[3]);
    w.z = pack_bf16x2(x[4], x[5]); w.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = w;
}

// Cache row of token t of (entry e, kv head h) for reading (block ids clamped
// into the pool), or -1 when `write` and the id lies outside it.
__device__ __forceinline__ long long cache_row(const CacheRows& c, int e, int h, int t, bool write) {
    if (!c.block_table) return ((long long)e * c.hkv + h) * c.s_cap + t;
    int blk = __ldg(c.block_table + (size_t)e * c.max_blocks + (t >> c.page_shift));
    if (write && (blk < 0 || blk >= c.num_blocks)) return -1;
    blk = min(max(blk, 0), c.num_blocks - 1);
    return ((((long long)blk * c.hkv + h) << c.page_shift)) + (t & ((1 << c.page_shift) - 1));
}

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kKvNT) ds_write_kv_kernel(const WriteArgs a, int split) {
    constexpr int kLanes = D / 16;          // lanes of one head's vector
    constexpr int kHeads = 32 / kLanes;     // heads a warp holds at a time
    const int lane = lane_id();
    const int sub = lane % kLanes, slot = lane / kLanes;
    const long long unit = (long long)blockIdx.x * (kKvNT / 32) + warp_id();  // (token, part of its heads)
    const long long token = unit / split;
    const int part = (int)(unit - token * split);
    if (token >= (long long)a.b * a.t) return;
    const int e = (int)(token / a.t), i = (int)(token - (long long)e * a.t);
    if (a.lens && i >= __ldg(a.lens + e)) return;
    const long long row = (long long)(a.starts ? __ldg(a.starts + e) : 0) + i;
    const bool row_ok = row >= 0 && row < a.rows;

    // this lane's chunks, and the rotation of its eight pairs
    int c0 = 16 * sub, c1 = 16 * sub + 8;
    const int half = a.rot_dim / 2;
    const bool turns = a.inv_freq != nullptr && 16 * sub < a.rot_dim;
    if (turns && !a.interleaved) { c0 = 8 * sub; c1 = half + 8 * sub; }
    float cs[8], sn[8];
    if (turns) {
        const double pos = a.positions ? (double)__ldg(a.positions + token) : (double)row;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // whole turns leave in 64 bits; what is left is exact to 2^-25 of a turn's half
            const double turn = pos * (double)__ldg(a.inv_freq + 8 * sub + j) * 0.15915494309189533577;
            sincospif(2.0f * (float)(turn - rint(turn)), &sn[j], &cs[j]);
        }
    }

    const int hq = a.q ? a.hq : 0, heads = hq + 2 * a.hkv;
    for (int h0 = part * kHeads; h0 < heads; h0 += split * kHeads) {
        const int h = h0 + slot;
        const bool live = h < heads;
        const int kind = h < hq ? 0 : h < hq + a.hkv ? 1 : 2;  // q, k, v
        const int hh = kind == 0 ? h : kind == 1 ? h - hq : h - hq - a.hkv;
        float x0[8], x1[8];
        if (live) {
            const T* src = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
            const long long bs = kind == 0 ? a.q_bs : kind == 1 ? a.k_bs : a.v_bs;
            const long long ts = kind == 0 ? a.q_ts : kind == 1 ? a.k_ts : a.v_ts;
            src += (long long)e * bs + (long long)i * ts + (long long)hh * D;
            load8<T>(x0, src + c0);
            load8<T>(x1, src + c1);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x0[j] = x1[j] = 0.f;
        }
        const T* w = static_cast<const T*>(kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x0[j], x0[j], fmaf(x1[j], x1[j], ss));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (live && w) {
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
            float w0[8], w1[8];
            load8<T>(w0, w + c0);
            load8<T>(w1, w + c1);
#pragma unroll
            for (int j = 0; j < 8; ++j) { x0[j] *= r * w0[j]; x1[j] *= r * w1[j]; }
        }
        if (live && turns && kind != 2) {
            if (!a.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p = x0[j], q = x1[j];
                    x0[j] = p * cs[j] - q * sn[j];
                    x1[j] = q * cs[j] + p * sn[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = x0[2 * j], q = x0[2 * j + 1], u = x1[2 * j], z = x1[2 * j + 1];
                    x0[2 * j] = p * cs[j] - q * sn[j];
                    x0[2 * j + 1] = q * cs[j] + p * sn[j];
                    x1[2 * j] = u * cs[j + 4] - z * sn[j + 4];
                    x1[2 * j + 1] = z * cs[j + 4] + u * sn[j + 4];
                }
            }
        }
        float amax = 0.f;
        if constexpr (Q8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max_nan(amax, max_nan(fabsf(x0[j]), fabsf(x1[j])));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        if (!live) continue;
        if (kind == 0) {
            T* out = static_cast<T*>(a.q_out) + (token * a.hq + hh) * D;
            store8(out + c0, x0);
            store8(out + c1, x1);
            continue;
        }
        if (!row_ok) continue;
        const long long r = cache_row(a.at, e, hh, (int)row, true);
        if (r < 0) continue;
        if constexpr (Q8) {
            float sc = max_nan(__fdiv_rn(amax, 448.f), 1.17549435e-38f);
            sc = fmaf(sc, 0.f, sc);  // an infinite scale becomes NaN: the row reads back as NaN
            const float rs = __frcp_rn(sc);
            uint32_t w0[2] = {0, 0}, w1[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                w0[j / 4] |= e4m3x2(divide(x0[j], sc, rs), divide(x0[j + 1], sc, rs)) << (8 * (j & 3));
                w1[j / 4] |= e4m3x2(divide(x1[j], sc, rs), divide(x1[j + 1], sc, rs)) << (8 * (j & 3));
            }
            uint8_t* out = static_cast<uint8_t*>(kind == 1 ? a.k_cache : a.v_cache) + r * D;
            *reinterpret_cast<uint2*>(out + c0) = make_uint2(w0[0], w0[1]);
            *reinterpret_cast<uint2*>(out + c1) = make_uint2(w1[0], w1[1]);
            if (sub == 0) (kind == 1 ? a.k_scale : a.v_scale)[r] = sc;
        } else {
            T* out = static_cast<T*>(kind == 1 ? a.k_cache : a.v_cache) + r * D;
            store8(out + c0, x0);
            store8(out + c1, x1);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kKvNT) ds_read_kv_kernel(const ReadArgs a) {
    const int per = a.d / 16;  // 16-code pieces of a row
    const long long pieces = (long long)a.b * a.hkv * a.s * per;
    const bool vals = blockIdx.y == 1;
    const uint8_t* src = static_cast<const uint8_t*>(vals ? a.v : a.k);
    const float* scale = vals ? a.v_scale : a.k_scale;
    T* dst = static_cast<T*>(vals ? a.v_out : a.k_out);
    for (long long p = (long long)blockIdx.x * kKvNT + threadIdx.x; p < pieces; p += (long long)gridDim.x * kKvNT) {
        const int c = (int)(p % per) * 16;
        const long long bhr = p / per;
        const int t = (int)(bhr % a.s);
        const long long bh = bhr / a.s;
        const int e = (int)(bh / a.hkv), h = (int)(bh % a.hkv);
        if (a.seq_lens && t >= __ldg(a.seq_lens + e)) continue;
        const long long r = cache_row(a.at, e, h, t, false);
        const uint4 w = ldg_stream16(src + r * a.d + c);
        const float sc = __ldg(scale + r);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
        float x[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = e4m3x2_to_f32(words[j / 2] >> (16 * (j & 1)) & 0xffffu);
            x[j / 4][2 * (j & 3)] = f.x * sc;
            x[j / 4][2 * (j & 3) + 1] = f.y * sc;
        }
        T* out = dst + (bh * a.s_out_cap + t) * a.d + c;
        store8(out, x[0]);
        store8(out + 8, x[1]);
    }
}

}  // namespace

cudaError_t launch_write_kv(const WriteArgs& a, cudaStream_t st) {
    const int heads = (a.q ? a.hq : 0) + 2 * a.hkv, per_warp = 32 / (a.d / 16);
    const long long tokens = (long long)a.b * a.t;
    // Few tokens: a token's heads go to several warps, until about 16 warps an
    // SM have work; many tokens: one warp a token, which computes its angles once.
    const long long want = (148 * 16 + tokens - 1) / tokens, most = (heads + per_warp - 1) / per_warp;
    const int split = (int)(want < most ? want : most);
    const long long warps = tokens * split;
    const unsigned grid = (unsigned)((warps + kKvNT / 32 - 1) / (kKvNT / 32));
#define DS_W(T_, D_, Q_) ds_write_kv_kernel<T_, D_, Q_><<<grid, kKvNT, 0, st>>>(a, split)
#define DS_WQ(T_, D_) (a.e4m3 ? (void)(DS_W(T_, D_, true)) : (void)(DS_W(T_, D_, false)))
    if (a.f32) a.d == 64 ? DS_WQ(float, 64) : DS_WQ(float, 128);
    else a.d == 64 ? DS_WQ(bf16_t, 64) : DS_WQ(bf16_t, 128);
#undef DS_WQ
#undef DS_W
    return cudaGetLastError();
}

cudaError_t launch_read_kv(const ReadArgs& a, cudaStream_t st) {
    const long long pieces = (long long)a.b * a.hkv * a.s * (a.d / 16);
    long long blocks = (pieces + kKvNT - 1) / kKvNT;
    if (blocks > 148 * 8) blocks = 148 * 8;
    const dim3 grid((unsigned)blocks, a.v ? 2 : 1);
    if (a.f32) ds_read_kv_kernel<float><<<grid, kKvNT, 0, st>>>(a);
    else ds_read_kv_kernel<bf16_t><<<grid, kKvNT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace ds
