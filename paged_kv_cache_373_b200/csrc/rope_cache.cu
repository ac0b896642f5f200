// rope_cache.cu -- pkv_qk_norm_rope_and_cache: per-head RMS norm of q and k,
// rotary embedding, and the write of k and v into their cache slots, in one
// pass over a step's projected rows.
//
// For a head row x of q or k:  y = x * rsqrt(mean(x^2) + eps) * w  (without
// weights y = x), then the first r = rotary_dim elements are turned pairwise by
// the angles of the token's position,
//   (a, b) -> (a cos - b sin, b cos + a sin),
// the pairs being (y[j], y[j + r/2]) or, interleaved, (y[2j], y[2j + 1]).  All in
// fp32 from the loaded values to the single rounding at the store; mean and
// rotation need every element of a row, so a row stays in registers.
//
// Bound: memory.  A row is read once and written once (~10 flops per element),
// the angles are r floats per token.  Layout: 8 elements per lane (16 bytes of a
// 16-bit row), so D / 8 neighbouring lanes hold a row: the norm is a shuffle
// reduction over them, and the partner element of a half-split pair is in the
// lane r / 16 further on.  A warp takes kRows rows per lane group of ONE token,
// so the token's angles are loaded once and used for all of them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

struct RopeParams {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // bytes between tokens
    void *q_out, *kc, *vc;
    const int64_t *slots, *positions;
    const float* cos_sin;                  // [max_position, rotary_dim]: cosines, then sines
    const void *qw, *kw;                   // [D] norm weights, or null
    const float *k_scale, *v_scale;
    int* err;
    int64_t num_tokens, num_slots, max_position;
    int hq, hkv, rotary, chunks;           // chunks: warps per token
    float eps;
};

// 8 consecutive elements of a row: 16 bytes (16-bit types) or 32 (f32).
template <typename T> struct Vec8 { uint4 w[sizeof(T) / 2]; };

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const uint8_t* p) {
    Vec8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void store8(uint8_t* p, const Vec8<T>& r) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
}
template <typename T>
__device__ __forceinline__ void widen8(const Vec8<T>& r, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * i] = __uint_as_float(r.w[i].x); x[4 * i + 1] = __uint_as_float(r.w[i].y);
            x[4 * i + 2] = __uint_as_float(r.w[i].z); x[4 * i + 3] = __uint_as_float(r.w[i].w);
        }
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<kB>(u[i]);
            x[2 * i] = f.x; x[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ Vec8<T> narrow8(const float (&x)[8]) {
    Vec8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        r.w[0] = make_uint4(pack2<kB>(x[0], x[1]), pack2<kB>(x[2], x[3]), pack2<kB>(x[4], x[5]), pack2<kB>(x[6], x[7]));
    }
    return r;
}
// 8 E4M3 codes of the fp32 quotients x / scale (RNE, saturating), as
// pkv_reshape_and_cache stores them.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
               ((uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16);
    return make_uint2(w[0], w[1]);
}

// kRows: rows per lane group and warp.  Rows of a token are numbered q heads,
// then k heads, then v heads.
template <typename T, int D, bool kFp8, bool kInter, int kRows>
__global__ void __launch_bounds__(256)
qk_norm_rope_kernel(const RopeParams p) {
    constexpr int G = D / 8;        // lanes per row
    constexpr int kGroups = 32 / G; // rows a warp holds side by side
    const int lane = threadIdx.x & 31, sub = lane % G, grp = lane / G;
    const int rows = p.hq + 2 * p.hkv;
    const int64_t total = p.num_tokens * p.chunks;
    const int half = p.rotary >> 4;  // lanes per half of the rotated part
    for (int64_t wid = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); wid < total; wid += (int64_t)gridDim.x * 8) {
        const int64_t t = wid / p.chunks;
        const int r0 = (int)(wid - t * p.chunks) * (kGroups * kRows) + grp;
        // the rows' loads go out before anything that depends on the slot
        Vec8<T> raw[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kGroups;
            const uint8_t* src;
            if (r < p.hq) src = static_cast<const uint8_t*>(p.q) + t * p.q_stride + (int64_t)r * (D * sizeof(T));
            else if (r < p.hq + p.hkv) src = static_cast<const uint8_t*>(p.k) + t * p.k_stride + (int64_t)(r - p.hq) * (D * sizeof(T));
            else src = static_cast<const uint8_t*>(p.v) + t * p.v_stride + (int64_t)(r - p.hq - p.hkv) * (D * sizeof(T));
            if (r < rows) raw[i] = load8<T>(src + sub * (8 * sizeof(T)));
            else raw[i] = Vec8<T>{};
        }
        const int64_t slot = __ldg(p.slots + t);
        if (slot < 0) continue;  // padding token
        if (slot >= p.num_slots) {
            if (lane == 0) raise_error(p.err, PKV_DEVERR_SLOT);
            continue;
        }
        float cs[8], sn[8];
        if (p.rotary > 0) {
            const int64_t pos = __ldg(p.positions + t);
            if (pos < 0 || pos >= p.max_position) {
                if (lane == 0) raise_error(p.err, PKV_DEVERR_POSITION);
                continue;
            }
            const float* row = p.cos_sin + pos * p.rotary;
            if (sub < 2 * half) {
                if constexpr (kInter) {  // pairs 4 sub .. 4 sub + 3 are in this lane
                    const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * sub));
                    const float4 s = __ldg(reinterpret_cast<const float4*>(row + 8 * half + 4 * sub));
                    cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
                    sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
                } else {                 // element j of either half takes angle j
                    const int j = 8 * (sub < half ? sub : sub - half);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 c = __ldg(reinterpret_cast<const float4*>(row + j) + e);
                        const float4 s = __ldg(reinterpret_cast<const float4*>(row + 8 * half + j) + e);
                        cs[4 * e] = c.x; cs[4 * e + 1] = c.y; cs[4 * e + 2] = c.z; cs[4 * e + 3] = c.w;
                        sn[4 * e] = s.x; sn[4 * e + 1] = s.y; sn[4 * e + 2] = s.z; sn[4 * e + 3] = s.w;
                    }
                }
            }
        }
        const bool turned = sub < 2 * half;
        // lane of the partner element (half-split pairs), and the sign of its sine
        const int partner = !turned ? lane : (sub < half ? lane + half : lane - half);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kGroups;
            const bool is_q = r < p.hq, is_v = r >= p.hq + p.hkv;
            float x[8];
            widen8<T>(raw[i], x);
            const void* wv = is_q ? p.qw : p.kw;
            if (p.qw) {  // every lane takes part in the shuffles; v rows keep their values
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
                if (!is_v) {
                    const float inv = rsqrtf(fmaf(ss, 1.f / D, p.eps));
                    float w[8];
                    widen8<T>(load8<T>(static_cast<const uint8_t*>(wv) + sub * (8 * sizeof(T))), w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
                }
            }
            if (p.rotary > 0) {
                if constexpr (kInter) {
                    if (turned && !is_v) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = x[2 * e], b = x[2 * e + 1];
                            x[2 * e] = a * cs[e] - b * sn[e];
                            x[2 * e + 1] = b * cs[e] + a * sn[e];
                        }
                    }
                } else {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(kFull, x[e], partner);
                    if (turned && !is_v) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = sub < half ? x[e] * cs[e] - y[e] * sn[e] : x[e] * cs[e] + y[e] * sn[e];
                    }
                }
            }
            if (r >= rows) continue;
            if (is_q) {
                store8<T>(static_cast<uint8_t*>(p.q_out) + ((t * p.hq + r) * D + 8 * sub) * (int64_t)sizeof(T), narrow8<T>(x));
                continue;
            }
            const int h = r - p.hq - (is_v ? p.hkv : 0);
            uint8_t* cache = static_cast<uint8_t*>(is_v ? p.vc : p.kc);
            const int64_t at = (slot * p.hkv + h) * D + 8 * sub;
            if constexpr (kFp8)
                *reinterpret_cast<uint2*>(cache + at) = quant8(x, __ldg(is_v ? p.v_scale : p.k_scale));
            else
                store8<T>(cache + at * (int64_t)sizeof(T), is_v ? raw[i] : narrow8<T>(x));
        }
    }
}

template <typename T, int D, bool kFp8, bool kInter, int kRows>
cudaError_t launch_rows(RopeParams& p, int sms, cudaStream_t st) {
    const int per_warp = (32 / (D / 8)) * kRows;
    p.chunks = (p.hq + 2 * p.hkv + per_warp - 1) / per_warp;
    const int64_t ctas = (p.num_tokens * p.chunks + 7) / 8;
    const int grid = (int)std::min<int64_t>(ctas, (int64_t)sms * 64);
    qk_norm_rope_kernel<T, D, kFp8, kInter, kRows><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int D, bool kFp8, bool kInter>
cudaError_t launch_rope(RopeParams& p, cudaStream_t st) {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // one row per lane group while the warps that gives do not fill the SMs,
    // four once they do
    const int64_t warps1 = p.num_tokens * ((p.hq + 2 * p.hkv + 32 / (D / 8) - 1) / (32 / (D / 8)));
    if (warps1 <= (int64_t)sms * 32) return launch_rows<T, D, kFp8, kInter, 1>(p, sms, st);
    return launch_rows<T, D, kFp8, kInter, 4>(p, sms, st);
}

template <typename T, int D>
cudaError_t launch_rope_t(RopeParams& p, bool fp8, bool inter, cudaStream_t st) {
    if (fp8) return inter ? launch_rope<T, D, true, true>(p, st) : launch_rope<T, D, true, false>(p, st);
    return inter ? launch_rope<T, D, false, true>(p, st) : launch_rope<T, D, false, false>(p, st);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_qk_norm_rope_and_cache(
    void* query_out, const void* query, int64_t query_stride, const void* key, int64_t key_stride,
    const void* value, int64_t value_stride, pkv_dtype dtype, void* key_cache, void* value_cache,
    pkv_dtype cache_dtype, const int64_t* slot_mapping, const int64_t* positions, const float* cos_sin,
    int64_t max_position, int rotary_dim, int interleaved, const void* q_weight, const void* k_weight,
    float eps, int64_t num_tokens, int64_t num_blocks, int block_size, int num_heads, int num_kv_heads,
    int head_dim, const float* k_scale, const float* v_scale, pkv_stream_t stream) {
    if (num_tokens < 0) return fail(PKV_EINVAL, "num_tokens < 0");
    if (num_blocks <= 0 || block_size <= 0) return fail(PKV_EINVAL, "num_blocks and block_size must be positive");
    if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads)
        return fail(PKV_EINVAL, "num_heads must be a positive multiple of num_kv_heads");
    if (head_dim != 64 && head_dim != 128) return fail(PKV_EUNSUPPORTED, "head_dim %d", head_dim);
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(PKV_EUNSUPPORTED, "rotary_dim %d: a multiple of 16 up to head_dim", rotary_dim);
    const int eb = dtype_bytes(dtype);
    if (eb == 0 || dtype_bytes(cache_dtype) == 0) return fail(PKV_EINVAL, "unknown dtype");
    const bool fp8 = cache_dtype == PKV_FP8_E4M3;
    if (dtype == PKV_FP8_E4M3) return fail(PKV_EUNSUPPORTED, "FP8 source");
    if (!fp8 && dtype != cache_dtype) return fail(PKV_EUNSUPPORTED, "non-FP8 caches need the source dtype");
    if (!q_weight != !k_weight) return fail(PKV_EINVAL, "q_weight and k_weight: both or neither");
    if (q_weight && !(eps >= 0.f && std::isfinite(eps))) return fail(PKV_EINVAL, "eps must be finite and not negative");
    if (rotary_dim > 0 && max_position <= 0) return fail(PKV_EINVAL, "max_position must be positive");
    const int64_t want[3] = {(int64_t)num_heads * head_dim, (int64_t)num_kv_heads * head_dim, (int64_t)num_kv_heads * head_dim};
    const int64_t have[3] = {query_stride, key_stride, value_stride};
    for (int i = 0; i < 3; ++i) {
        if (have[i] < want[i]) return fail(PKV_EINVAL, "token stride %lld < %lld elements", (long long)have[i], (long long)want[i]);
        if (have[i] * eb % 16) return fail(PKV_EINVAL, "token strides must be multiples of 16 bytes");
    }
    if (num_tokens == 0) return PKV_OK;
    if (!query_out || !query || !key || !value || !key_cache || !value_cache || !slot_mapping)
        return fail(PKV_EINVAL, "null pointer");
    if (rotary_dim > 0 && (!positions || !cos_sin)) return fail(PKV_EINVAL, "rotary_dim > 0 needs positions and cos_sin");
    if (fp8 && (!k_scale || !v_scale)) return fail(PKV_EINVAL, "FP8 cache needs k_scale and v_scale");
    if (!aligned16(query_out) || !aligned16(query) || !aligned16(key) || !aligned16(value) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned16(cos_sin) || !aligned16(q_weight) || !aligned16(k_weight))
        return fail(PKV_EINVAL, "buffers must be 16-byte aligned");
    if (query == query_out && query_stride != want[0])
        return fail(PKV_EINVAL, "query_out in place of a query with another token stride");
    int* err = device_error_word();
    if (!err) return fail(PKV_ECUDA, "device error word unavailable");
    RopeParams p{};
    p.q = query; p.k = key; p.v = value;
    p.q_stride = query_stride * eb; p.k_stride = key_stride * eb; p.v_stride = value_stride * eb;
    p.q_out = query_out; p.kc = key_cache; p.vc = value_cache;
    p.slots = slot_mapping; p.positions = positions; p.cos_sin = cos_sin;
    p.qw = q_weight; p.kw = k_weight; p.k_scale = k_scale; p.v_scale = v_scale;
    p.err = err;
    p.num_tokens = num_tokens; p.num_slots = num_blocks * block_size; p.max_position = max_position;
    p.hq = num_heads; p.hkv = num_kv_heads; p.rotary = rotary_dim; p.eps = eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool inter = interleaved != 0;
    cudaError_t e;
    switch (dtype) {
    case PKV_F32:
        e = head_dim == 64 ? launch_rope_t<float, 64>(p, fp8, inter, st) : launch_rope_t<float, 128>(p, fp8, inter, st);
        break;
    case PKV_F16:
        e = head_dim == 64 ? launch_rope_t<__half, 64>(p, fp8, inter, st) : launch_rope_t<__half, 128>(p, fp8, inter, st);
        break;
    default:
        e = head_dim == 64 ? launch_rope_t<__nv_bfloat16, 64>(p, fp8, inter, st)
                           : launch_rope_t<__nv_bfloat16, 128>(p, fp8, inter, st);
        break;
    }
    if (e != cudaSuccess) return fail(PKV_ECUDA, "qk_norm_rope launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}
