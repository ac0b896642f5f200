// prefill.cuh -- what the two chunked-prefill kernels share: the parameters, the
// geometry of a 128-row unit and the host checks (prefill.cu).
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr uint64_t kPfWaitNs = 200000000ull;  // limit of every wait

struct PrefillParams {
    void* out;
    const int32_t* tables;
    const int32_t* seq_lens;
    const int32_t* qstart;
    int* err;
    int64_t num_blocks, num_tokens;  // num_tokens: rows of query and out
    int num_seqs, num_heads, num_kv_heads, g, mbps, bs;
    float scale_log2;
    uint64_t wait_ns;  // limit of every wait (kPfWaitNs)
    int stop_tile;     // < 0; a test of the timeout path sets k >= 0: K/V tiles k, k+1, ... are never copied
};

// Rows of sequence s's chunk; -1 where query_start decreases or leaves the rows of the
// call (nothing may be written for it).
__device__ __forceinline__ int chunk_rows(const PrefillParams& p, int s) {
    const int q0 = __ldg(p.qstart + s), q1 = __ldg(p.qstart + s + 1);
    if (q1 == q0) return 0;
    return q0 >= 0 && q1 > q0 && q1 <= p.num_tokens ? q1 - q0 : -1;
}

// Validate the arguments of a prefill call and fill the kernel parameters and
// the grid: one CTA per kv head and pair of 128-row units, an upper bound taken
// from the number of rows (0: nothing to launch).  Disarms a timeout test.
pkv_status prefill_prepare(PrefillParams* p, int64_t* grid, void* out, const void* query, pkv_dtype q_dtype,
                           const void* key_cache, const void* value_cache, pkv_dtype cache_dtype,
                           const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                           const int32_t* query_start, int num_seqs, int64_t num_query_tokens, int num_heads,
                           int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale);

}  // namespace pkv
