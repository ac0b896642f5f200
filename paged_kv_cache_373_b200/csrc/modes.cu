// modes.cu -- pkv_paged_attention_decode_scoremod and
// pkv_paged_attention_decode_weights: the decode pass with modified scores, and
// the decode pass that also accumulates every cached token's attention weight.
// Both are variants of pkv_decode_kernel (paged_attention.cuh) and share its
// split of all tiles over the warps of a persistent grid and its exact merge.
//
// Bound: memory for large batches, the chain of dependent loads (lengths, table,
// K and V, partial results) for small ones.  With modified scores: 128 sequences of
// 64 to 8192 tokens, 32 / 8 heads of 128, bf16, capped: 141 us, 6250 GB/s (the K and V
// bytes once); 3 sequences of up to 301 tokens 6.0 us; 16 FP8 sequences with a window
// of 4096 and 64 kept tokens 35 us, 3900 GB/s, of which 25 us are the tile loop (5400
// GB/s) and the rest its start and the merge.  With weights: 64 sequences of 64 to
// 8192 tokens 87 us, 5150 GB/s: the decode pass some 75, the merge 4, the weights pass 8 (its
// scores, 4 bytes per q head and token, written once and read once, mostly in L2);
// 5 sequences of up to 777 tokens 7.4 us (f16: 0.2 of them for its second sum per row).
#include <cfloat>
#include <cmath>

#include "attn_launch.cuh"
#include "pkv_internal.h"

namespace pkv {

pkv_status score_cap(float softcap, float* cap2, float* inv_cap2) {
    *cap2 = *inv_cap2 = 0.f;
    if (softcap == 0.f) return PKV_OK;
    const double c = (double)softcap * 1.4426950408889634;
    if (!(c > 0.0) || c > (double)FLT_MAX || 1.0 / c > (double)FLT_MAX)
        return fail(PKV_EINVAL, "softcap must be 0 or positive, finite and not denormal");
    *cap2 = (float)c;
    *inv_cap2 = (float)(1.0 / c);
    return PKV_OK;
}

namespace {

// The weights pass of large batches, after their merge pass has written every lse.
__global__ void __launch_bounds__(kWeightThreads)
pkv_weights_kernel(const DecodeParams p, const WeightsArg a) {
    const WaitPrimaryAtExit<true> wait_at_exit;
    const Lens<false> ln{p.seq_lens, nullptr, p.num_seqs, p.num_kv_heads, p.max_blocks_per_seq * p.block_size};
    constexpr int kTokens = kWeightThreads * 4;
    int64_t W, tb, te;
    Walk<kTokens> w;
    auto share = [&](int64_t total) {
        const int64_t each = quot(total + gridDim.x - 1, gridDim.x);
        tb = min(total, blockIdx.x * each);
        te = min(total, tb + each);
        return tb;
    };
    if (p.num_seqs <= 32 * kScanPerLane) {
        bool bad;  // (the decode pass has raised it)
        const SeqHit hit = lane_scan<kTokens, kScanPerLane>(ln, share, &W, &bad);
        w.init<true>(ln, tb, te, hit);
    } else {
        share(W = total_tiles<kTokens>(ln));
        w.init(ln, tb, te);
    }
    if (tb >= te) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (; !w.done; w.advance(ln))
        weights_item<kWeightThreads>(p, a, w, a.lse + (int64_t)w.s * p.num_heads + (int64_t)w.j * p.g);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct WeightsLayout {
    size_t seg_mu, lse, scores, total;
};
bool weights_layout(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int64_t max_tokens, int num_ctas,
                    WeightsLayout* l) {
    const size_t dec = decode_workspace_bytes(num_seqs, num_heads, num_kv_heads, head_dim, num_ctas);
    if (dec == 0 || max_tokens <= 0 || max_tokens > 0x7fffffffLL) return false;
    const size_t rows = (size_t)num_seqs * num_heads;
    l->seg_mu = align256(dec);
    l->lse = l->seg_mu + align256(decode_segment_rows(num_seqs, num_heads, num_kv_heads, head_dim, num_ctas) *
                                  sizeof(float2));
    l->scores = l->lse + align256(rows * sizeof(float));
    l->total = l->scores + rows * (size_t)max_tokens * sizeof(float);
    return true;
}

}  // namespace

pkv_status launch_weights_pass(const DecodeParams& p, const WeightsArg& a, int grid, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)weight_ctas(p, grid, kWeightThreads));
    cfg.blockDim = dim3(kWeightThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, pkv_weights_kernel, p, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "weights launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_paged_attention_decode_scoremod(
    void* out, const void* query, pkv_dtype q_dtype, const void* key_cache, const void* value_cache,
    pkv_dtype cache_dtype, const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
    int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale,
    float softcap, int window, const float* alibi_slopes, const int32_t* prefix_lens, const float* k_scale,
    const float* v_scale, void* workspace, size_t workspace_bytes, int num_ctas, pkv_stream_t stream) {
    ModArg m{alibi_slopes, prefix_lens, 0.f, 0.f, window};
    pkv_status st = score_cap(softcap, &m.cap2, &m.inv_cap2);
    if (st != PKV_OK) return st;
    if (window < 0) return fail(PKV_EINVAL, "window < 0");
    DecodeParams p;
    DecodeLauncher plain;
    int grid = 0;
    st = decode_prepare(&p, &plain, &grid, out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables,
                        max_blocks_per_seq, seq_lens, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, scale, k_scale, v_scale, workspace, workspace_bytes, num_ctas);
    if (st != PKV_OK || num_seqs == 0) return st;
    DecodeLaunchArgs a{&p, grid};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (cache_dtype) {
    case PKV_F32: return launch_mod_f32(a, m, head_dim, s);
    case PKV_F16: return launch_mod_f16(a, m, head_dim, s);
    case PKV_BF16: return launch_mod_bf16(a, m, head_dim, s);
    default: return launch_mod_fp8(a, m, q_dtype == PKV_BF16, s);
    }
}

extern "C" size_t pkv_paged_attention_weights_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                                              int head_dim, int64_t max_tokens, int num_ctas) {
    WeightsLayout l;
    return weights_layout(num_seqs, num_heads, num_kv_heads, head_dim, max_tokens, num_ctas, &l) ? l.total : 0;
}

extern "C" pkv_status pkv_paged_attention_decode_weights(
    void* out, float* weights_out, const float* weights_in, int64_t weight_len, const void* query, pkv_dtype q_dtype,
    const void* key_cache, const void* value_cache, pkv_dtype cache_dtype, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* seq_lens, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
    int block_size, int64_t num_blocks, float scale, const float* k_scale, const float* v_scale, void* workspace,
    size_t workspace_bytes, int num_ctas, pkv_stream_t stream) {
    if (weight_len <= 0) return fail(PKV_EINVAL, "weight_len must be positive");
    if (num_seqs > 0 && !weights_out) return fail(PKV_EINVAL, "null pointer");
    const double weight_bytes = 4.0 * num_seqs * num_kv_heads * weight_len;
    if (weights_in && weights_in != weights_out &&
        overlap({"weights_in", weights_in, weight_bytes}, {"weights_out", weights_out, weight_bytes}))
        return fail(PKV_EINVAL, "weights_in overlaps weights_out");
    DecodeParams p;
    DecodeLauncher plain;
    int grid = 0;
    pkv_status st = decode_prepare(&p, &plain, &grid, out, query, q_dtype, key_cache, value_cache, cache_dtype,
                                   block_tables, max_blocks_per_seq, seq_lens, num_seqs, num_heads, num_kv_heads,
                                   head_dim, block_size, num_blocks, scale, k_scale, v_scale, workspace,
                                   workspace_bytes, num_ctas);
    if (st != PKV_OK || num_seqs == 0) return st;
    const int64_t max_tokens = (int64_t)max_blocks_per_seq * block_size;
    WeightsLayout l;
    if (!weights_layout(num_seqs, num_heads, num_kv_heads, head_dim, max_tokens, num_ctas, &l))
        return fail(PKV_ECUDA, "cannot size the grid");
    if (workspace_bytes < l.total)
        return fail(PKV_EINVAL, "workspace too small: %zu < %zu bytes", workspace_bytes, l.total);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const WeightsArg w{reinterpret_cast<float*>(ws + l.scores), reinterpret_cast<float*>(ws + l.lse),
                       reinterpret_cast<float2*>(ws + l.seg_mu), max_tokens, weights_in, weights_out, weight_len,
                       weight_len % 4 == 0 && aligned16(weights_in) && aligned16(weights_out)};
    DecodeLaunchArgs a{&p, grid};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (cache_dtype) {
    case PKV_F32: return launch_scores_f32(a, w, head_dim, s);
    case PKV_F16: return launch_scores_f16(a, w, head_dim, s);
    case PKV_BF16: return launch_scores_bf16(a, w, head_dim, s);
    default: return launch_scores_fp8(a, w, q_dtype == PKV_BF16, s);
    }
}
