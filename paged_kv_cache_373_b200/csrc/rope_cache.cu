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
// the angles are r floats per token.  Layout: D / 8 neighbouring lanes hold a row,
// a lane two runs of 4 elements: of the rotated part the run at 4 l and its partners
// at r/2 + 4 l (half-split pairs) or at 8 l and 8 l + 4 (interleaved ones), so every pair
// is in one lane and a lane needs 4 angles; the norm is a shuffle reduction.  (With
// 8 neighbouring elements per lane the partners came by 8 shuffles a row and a lane
// loaded 8 angles: 37.8 against 33.4 us for 8192 tokens of 16 + 8 + 8 heads of 128,
// bf16.)
// A warp's item is kRows rows per lane group of ONE token and one kind (q, k or v),
// so the token's angles are loaded once for all of them and nothing asks per row
// (167 instructions a row and 33.4 us before, 25.6 us since; 24.7 with the fourth CTA:
// 5600 GB/s, 86 % of the measured copy rate).
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
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    void *q_out, *kc, *vc;
    const int64_t *slots, *positions;
    const float* cos_sin;                  // [max_position, rotary_dim]: cosines, then sines
    const void *qw, *kw;                   // [D] norm weights, or null
    const float *k_scale, *v_scale;
    int* err;
    int64_t num_tokens, num_slots, max_position;
    int hq, hkv, rotary;
    float eps;
};

// Two runs of 4 elements: 8 bytes each (16-bit types) or 16 (f32).
template <typename T> struct Runs {
    using V = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
    V a, b;
};
template <typename T>
__device__ __forceinline__ Runs<T> load_runs(const T* row, int oa, int ob) {
    using V = typename Runs<T>::V;
    return Runs<T>{*reinterpret_cast<const V*>(row + oa), *reinterpret_cast<const V*>(row + ob)};
}
template <typename T>
__device__ __forceinline__ void store_runs(T* row, int oa, int ob, const Runs<T>& r) {
    using V = typename Runs<T>::V;
    *reinterpret_cast<V*>(row + oa) = r.a;
    *reinterpret_cast<V*>(row + ob) = r.b;
}
template <typename T>
__device__ __forceinline__ void widen4(const uint2& w, float* x) {
    constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
    const float2 f = unpack2<kB>(w.x), g = unpack2<kB>(w.y);
    x[0] = f.x; x[1] = f.y; x[2] = g.x; x[3] = g.y;
}
template <typename T>
__device__ __forceinline__ void widen4(const uint4& w, float* x) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
}
template <typename T>
__device__ __forceinline__ void widen(const Runs<T>& r, float (&x)[8]) {
    widen4<T>(r.a, x);
    widen4<T>(r.b, x + 4);
}
template <typename T>
__device__ __forceinline__ typename Runs<T>::V narrow4(const float* x) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        return make_uint2(pack2<kB>(x[0], x[1]), pack2<kB>(x[2], x[3]));
    }
}
// 4 E4M3 codes of the fp32 quotients x / scale (RNE, saturating), as
// pkv_reshape_and_cache stores them.
__device__ __forceinline__ uint32_t quant4(const float* x, float scale) {
    return (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
           ((uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16);
}

// CTAs per SM of the persistent grid: 4 (64 registers) for plain 16-bit rows, 24.7 us for
// the 8192 tokens above (3: 25.6); FP8 codes and f32 rows need more registers, 3 (1023
// tokens of 64 + 8 + 8 heads into FP8 7.1 us, with 4 7.5).
template <typename T, bool kFp8> constexpr int kRopeCtas = sizeof(T) == 2 && !kFp8 ? 4 : 3;

enum class Rows { kQ, kK, kV };

// One item: up to kRows rows per lane group of one token, all q, all k or all v
// rows (so that nothing in the loop asks which).  src, dst: the item's first row of
// this lane group; left: rows from there on; w: the lane's norm weights, or unused.
template <typename T, int D, bool kFp8, bool kInter, int kRows, Rows kKind>
__device__ __forceinline__ void rope_item(const RopeParams& p, const T* src, void* dst, int left, int64_t pos,
                                          const Runs<T>& wr, bool norm, bool turned, int oa, int ob) {
    constexpr int G = D / 8, kStep = 32 / G * D;  // elements between a lane group's rows
    constexpr bool kCodes = kFp8 && kKind != Rows::kQ;
    Runs<T> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) raw[i] = i * (32 / G) < left ? load_runs(src + i * kStep, oa, ob) : Runs<T>{};
    float c[4] = {}, d[4] = {}, w[8];  // the lane's 4 angles and 8 norm weights
    if constexpr (kKind != Rows::kV) {
        if (turned) {
            const float* row = p.cos_sin + pos * p.rotary + (kInter ? oa / 2 : oa);
            const float4 cs = __ldg(reinterpret_cast<const float4*>(row));
            const float4 sn = __ldg(reinterpret_cast<const float4*>(row + p.rotary / 2));
            c[0] = cs.x; c[1] = cs.y; c[2] = cs.z; c[3] = cs.w;
            d[0] = sn.x; d[1] = sn.y; d[2] = sn.z; d[3] = sn.w;
        }
        widen(wr, w);
    }
    float scale = 1.f;
    if constexpr (kCodes) scale = __ldg(kKind == Rows::kK ? p.k_scale : p.v_scale);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        Runs<T> r = raw[i];
        float x[8];
        if constexpr (kKind != Rows::kV || kCodes) widen(r, x);
        if constexpr (kKind != Rows::kV) {
            if (norm) {  // warp-uniform: every lane takes part in the shuffles
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
                const float inv = rsqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
            }
            if (turned) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int ia = kInter ? 2 * e : e, ib = kInter ? 2 * e + 1 : e + 4;
                    const float a = x[ia], b = x[ib];
                    x[ia] = a * c[e] - b * d[e];
                    x[ib] = b * c[e] + a * d[e];
                }
            }
            if constexpr (!kCodes) r = Runs<T>{narrow4<T>(x), narrow4<T>(x + 4)};
        }
        if (i * (32 / G) < left) {
            if constexpr (kCodes) {
                uint8_t* row = static_cast<uint8_t*>(dst) + i * kStep;
                *reinterpret_cast<uint32_t*>(row + oa) = quant4(x, scale);
                *reinterpret_cast<uint32_t*>(row + ob) = quant4(x + 4, scale);
            } else {
                store_runs(static_cast<T*>(dst) + i * kStep, oa, ob, r);
            }
        }
    }
}

template <typename T, int D, bool kFp8, bool kInter, int kRows>
__global__ void __launch_bounds__(256, (kRopeCtas<T, kFp8>))
qk_norm_rope_kernel(const RopeParams p) {
    constexpr int G = D / 8;                  // lanes per row
    constexpr int kPer = 32 / G * kRows;      // rows per item
    using CT = typename std::conditional<kFp8, uint8_t, T>::type;
    const int lane = threadIdx.x & 31, sub = lane % G, grp = lane / G;
    const bool turned = 8 * sub < p.rotary;
    // the lane's runs: of the rotated part, or 8 neighbours behind it
    const int oa = !kInter && turned ? 4 * sub : 8 * sub, ob = !kInter && turned ? p.rotary / 2 + 4 * sub : 8 * sub + 4;
    // a token's items: iq of q rows, ik of k rows, ik of v rows
    const int iq = (p.hq + kPer - 1) / kPer, ik = (p.hkv + kPer - 1) / kPer, items = iq + 2 * ik;
    const int64_t step = (int64_t)gridDim.x * 8, wid = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    int64_t t = wid / items;
    int it = (int)(wid - t * items);
    const int64_t dt = step / items;
    const int di = (int)(step - dt * items);
    if (t >= p.num_tokens) return;
    // the norm weights of this lane's elements, for q and k rows
    const bool norm = p.qw != nullptr;
    Runs<T> wq{}, wk{};
    if (norm) {
        wq = load_runs(static_cast<const T*>(p.qw), oa, ob);
        wk = load_runs(static_cast<const T*>(p.kw), oa, ob);
    }
    // slot and position one item ahead: the angles are then one load away
    int64_t slot = __ldg(p.slots + t), pos = p.rotary > 0 ? __ldg(p.positions + t) : 0;
    while (true) {
        int64_t nt = t + dt;
        int ni = it + di;
        if (ni >= items) { ni -= items; ++nt; }
        const bool more = nt < p.num_tokens;
        int64_t next_slot = 0, next_pos = 0;
        if (more) {
            next_slot = __ldg(p.slots + nt);
            if (p.rotary > 0) next_pos = __ldg(p.positions + nt);
        }
        if (slot >= p.num_slots) {
            if (lane == 0) raise_error(p.err, PKV_DEVERR_SLOT);
        } else if (slot >= 0 && p.rotary > 0 && (pos < 0 || pos >= p.max_position)) {
            if (lane == 0) raise_error(p.err, PKV_DEVERR_POSITION);
        } else if (slot >= 0) {  // below 0: a padding token
            if (it < iq) {
                const int r = it * kPer + grp;
                rope_item<T, D, kFp8, kInter, kRows, Rows::kQ>(
                    p, static_cast<const T*>(p.q) + t * p.q_stride + r * D,
                    static_cast<T*>(p.q_out) + (t * p.hq + r) * D, p.hq - r, pos, wq, norm, turned, oa, ob);
            } else if (it < iq + ik) {
                const int r = (it - iq) * kPer + grp;
                rope_item<T, D, kFp8, kInter, kRows, Rows::kK>(
                    p, static_cast<const T*>(p.k) + t * p.k_stride + r * D,
                    static_cast<CT*>(p.kc) + (slot * p.hkv + r) * D, p.hkv - r, pos, wk, norm, turned, oa, ob);
            } else {
                const int r = (it - iq - ik) * kPer + grp;
                rope_item<T, D, kFp8, kInter, kRows, Rows::kV>(
                    p, static_cast<const T*>(p.v) + t * p.v_stride + r * D,
                    static_cast<CT*>(p.vc) + (slot * p.hkv + r) * D, p.hkv - r, pos, wk, norm, turned, oa, ob);
            }
        }
        if (!more) return;
        t = nt; it = ni; slot = next_slot; pos = next_pos;
    }
}

template <typename T, int D, bool kFp8, bool kInter, int kRows>
cudaError_t launch_rows(RopeParams& p, int sms, cudaStream_t st) {
    const int per = 32 / (D / 8) * kRows;  // rows per warp and item
    const int64_t items = p.num_tokens * ((p.hq + per - 1) / per + 2 * ((p.hkv + per - 1) / per));
    const int64_t ctas = (items + 7) / 8;
    const int grid = (int)std::min<int64_t>(ctas, (int64_t)sms * kRopeCtas<T, kFp8>);
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

// Whether n rows of `row` bytes, `stride` apart, meet the n contiguous rows of `out_row`
// bytes at `out`.
bool rows_overlap(const void* rows, int64_t stride, int64_t row, const void* out, int64_t out_row, int64_t n) {
    const double d = (double)(intptr_t)((uintptr_t)out - (uintptr_t)rows);  // out, seen from the first row
    // the first row that ends behind out's start
    const double i = d < (double)row ? 0.0 : std::floor((d - (double)row) / (double)stride) + 1.0;
    return i < (double)n && i * (double)stride < d + (double)out_row * (double)n;
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
    // query_out apart from the rows that are read (or exactly query, row by row)
    const void* rows[3] = {query, key, value};
    const char* names[3] = {"query", "key", "value"};
    for (int i = query == query_out ? 1 : 0; i < 3; ++i)
        if (rows_overlap(rows[i], have[i] * eb, want[i] * eb, query_out, want[0] * eb, num_tokens))
            return fail(PKV_EINVAL, "query_out overlaps %s", names[i]);
    int* err = device_error_word();
    if (!err) return fail(PKV_ECUDA, "device error word unavailable");
    RopeParams p{};
    p.q = query; p.k = key; p.v = value;
    p.q_stride = query_stride; p.k_stride = key_stride; p.v_stride = value_stride;
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
