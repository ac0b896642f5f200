// evict.cu -- pkv_evict_tokens: cache eviction by accumulated attention weight.
// Per (sequence, kv head) with more tokens than the budget, the last `recent`
// tokens and the heaviest of the others stay, in ascending order, and their K/V
// rows move to the first `budget` slots of a new block table.
//
// Two kernels.
//   select: one CTA per (sequence, kv head) finds the budget's threshold by radix
//     selection on the weights' bits (11 + 11 + 10 bits, a shared-memory histogram
//     a pass), then numbers the kept tokens in order by ballots and one scan.  A row
//     of up to 16384 weights is loaded once and stays in registers (a longer one is
//     read again each pass).  Integer work only, so the result does not depend on
//     any order.  Bound: the latency of its barriers and shared-memory atomics.
//   gather: one CTA per destination block copies its rows, 16 bytes per thread and
//     access, K and V in flight together.  Bound: memory -- every kept row is read
//     and written once; a row is at least one 64-byte run.
// The source and the destination are different blocks, so nothing is moved onto
// rows still to be read, blocks shared with other sequences stay as they are, and
// the copy needs no order.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

struct EvictParams {
    uint8_t *kc, *vc;
    const int32_t *tables, *new_tables, *seq_lens;
    const float* weights;
    int32_t* new_lens;
    float* new_weights;
    int32_t* kept;
    int* err;
    int64_t weight_len, new_weight_len, num_blocks;
    int num_seqs, hkv, mbps, new_mbps, bs, budget, recent, row_bytes;
};

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeys = 16;                           // weights a thread holds
constexpr int kBatch = kSelThreads * kKeys;         // tokens the CTA holds at once
constexpr int kRuns = kSelWarps * kKeys;            // runs of 32 neighbouring tokens in a batch

// Order-preserving map of a weight to an unsigned key; NaN is the lowest, -0 is +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The attended length of sequence s that the call works on, and whether its
// tables and rows hold it.
__device__ __forceinline__ int evict_len(const EvictParams& p, int s, bool* bad) {
    const int raw = __ldg(p.seq_lens + s);
    const int64_t cap = min((int64_t)p.mbps * p.bs, p.weight_len);
    const int L = raw < 0 ? 0 : (int)min((int64_t)raw, cap);
    *bad = L != raw || min(L, p.budget) > p.new_weight_len ||
           (L > p.budget && (int64_t)p.new_mbps * p.bs < p.budget);
    return L;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int hist[kBins];
    __shared__ int wsum[kSelWarps];
    __shared__ int run_gt[kRuns], run_eq[kRuns];
    __shared__ uint32_t sh_digit;
    __shared__ int sh_left;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t u = blockIdx.x;
    const int s = (int)(u / p.hkv), h = (int)(u % p.hkv);
    bool bad;
    const int L = evict_len(p, s, &bad);
    if (h == 0 && tid == 0) {
        if (bad) raise_error(p.err, PKV_DEVERR_SEQ_LEN);
        p.new_lens[s] = min(L, p.budget);
    }
    const float* w = p.weights + u * p.weight_len;
    float* nw = p.new_weights + u * p.new_weight_len;
    int32_t* kept = p.kept + u * p.budget;
    auto keep = [&](int j, int t) {
        kept[j] = t;
        if (j < p.new_weight_len) nw[j] = w[t];
    };
    if (L <= p.budget) {  // everything stays where it is
        for (int j = tid; j < p.budget; j += kSelThreads) {
            if (j < L) keep(j, j);
            else kept[j] = -1;
        }
        return;
    }
    const int m = L - p.recent;       // tokens to choose from
    const int c = p.budget - p.recent;  // of which c stay (0 <= c < m)
    for (int t = m + tid; t < L; t += kSelThreads) keep(c + t - m, t);
    if (c == 0) return;

    // the weights of a batch, all loads in flight; a row that fits one batch is
    // loaded once and stays in registers through the passes
    uint32_t key[kKeys];
    auto load = [&](int base) {
        float x[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int t = base + i * kSelThreads + tid;
            x[i] = t < m ? w[t] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kKeys; ++i) key[i] = weight_key(x[i]);
    };
    const bool one = m <= kBatch;
    if (one) load(0);

    // ---- the c-th largest key: digit by digit from the top
    uint32_t prefix = 0;
    int left = c;  // rank still to find among the keys that share the prefix
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = d == 0 ? 0u : 0xffffffffu << (kShift[d] + kBits[d]);
        for (int base = 0; base < m; base += kBatch) {
            if (!one) load(base);
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                const uint32_t k = key[i];
                if (base + i * kSelThreads + tid < m && (k & mask) == prefix)
                    atomicAdd(&hist[(k >> kShift[d]) & ((1u << kBits[d]) - 1)], 1);
            }
        }
        __syncthreads();
        // thread i holds bins kBins-1-2i and kBins-2-2i: counts from the top down
        const int hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
        int incl = hi + lo;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        if (warp == 0) {
            const int v = wsum[lane];
            int x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            wsum[lane] = x - v;
        }
        __syncthreads();
        const int before = wsum[warp] + incl - hi - lo;  // keys in higher bins
        if (left > before && left <= before + hi + lo) {
            const bool first = left <= before + hi;
            sh_digit = (uint32_t)(kBins - 1 - 2 * tid - (first ? 0 : 1));
            sh_left = left - before - (first ? 0 : hi);
        }
        __syncthreads();
        prefix |= sh_digit << kShift[d];
        left = sh_left;
    }
    // every key above `prefix` stays, and the first `left` of those equal to it

    // ---- number the kept tokens in order: the ballots of a batch's runs of 32
    // tokens (run i * kSelWarps + warp), a scan over the runs, and the totals so far
    int gt0 = 0, eq0 = 0;
    const unsigned below = (1u << lane) - 1;
    for (int base = 0; base < m; base += kBatch) {
        if (!one) load(base);
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const bool in = base + i * kSelThreads + tid < m;
            const unsigned bg = __ballot_sync(kFull, in && key[i] > prefix);
            const unsigned be = __ballot_sync(kFull, in && key[i] == prefix);
            if (lane == 0) {
                run_gt[i * kSelWarps + warp] = __popc(bg);
                run_eq[i * kSelWarps + warp] = __popc(be);
            }
        }
        __syncthreads();
        if (warp < 2) {  // exclusive scan of kRuns counts, kKeys per lane; warp 0: gt, warp 1: eq
            int* run = warp ? run_eq : run_gt;
            int v[kKeys], sum = 0;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                v[i] = run[lane * kKeys + i];
                sum += v[i];
            }
            int x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) wsum[warp] = x;
            x -= sum;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                run[lane * kKeys + i] = x;
                x += v[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int t = base + i * kSelThreads + tid;
            const bool is_gt = t < m && key[i] > prefix, is_eq = t < m && key[i] == prefix;
            const unsigned bg = __ballot_sync(kFull, is_gt), be = __ballot_sync(kFull, is_eq);
            const int g = gt0 + run_gt[i * kSelWarps + warp] + __popc(bg & below);
            const int e = eq0 + run_eq[i * kSelWarps + warp] + __popc(be & below);
            if (is_gt || (is_eq && e < left)) keep(g + min(e, left), t);
        }
        gt0 += wsum[0];
        eq0 += wsum[1];
        __syncthreads();
    }
}

constexpr int kGatThreads = 256;

// CTA: destination block b of sequence s.  Chunk c of row (slot, head): the
// destination is one contiguous run, the sources rows of the old blocks.
__global__ void __launch_bounds__(kGatThreads)
evict_gather_kernel(const EvictParams p, int nblk) {
    const int s = (int)(blockIdx.x / nblk), b = (int)(blockIdx.x % nblk);
    bool bad;
    const int L = evict_len(p, s, &bad);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (L <= p.budget) return;
    const int dst = __ldg(p.new_tables + (int64_t)s * p.new_mbps + b);
    if (dst < 0 || dst >= p.num_blocks) {
        if (threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const int cpr = p.row_bytes / 16;
    const int slots = min(p.bs, p.budget - b * p.bs);
    const int chunks = slots * p.hkv * cpr;
    const int32_t* table = p.tables + (int64_t)s * p.mbps;
    const int64_t dbase = (int64_t)dst * p.bs * p.hkv * p.row_bytes;
    for (int i = threadIdx.x; i < chunks; i += kGatThreads) {
        const int row = i / cpr, c = i - row * cpr;
        const int slot = row / p.hkv, h = row - slot * p.hkv;
        const int t = p.kept[((int64_t)s * p.hkv + h) * p.budget + b * p.bs + slot];
        const int src = __ldg(table + t / p.bs);
        if (src < 0 || src >= p.num_blocks) {
            if (c == 0) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
            continue;
        }
        const int64_t from = (((int64_t)src * p.bs + t % p.bs) * p.hkv + h) * p.row_bytes + 16 * c;
        const int64_t to = dbase + (int64_t)i * 16;
        const uint4 k = *reinterpret_cast<const uint4*>(p.kc + from);
        const uint4 v = *reinterpret_cast<const uint4*>(p.vc + from);
        *reinterpret_cast<uint4*>(p.kc + to) = k;
        *reinterpret_cast<uint4*>(p.vc + to) = v;
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_evict_tokens(void* key_cache, void* value_cache, pkv_dtype cache_dtype,
                                       const int32_t* block_tables, int max_blocks_per_seq,
                                       const int32_t* seq_lens, const float* weights, int64_t weight_len,
                                       const int32_t* new_block_tables, int new_max_blocks_per_seq,
                                       int32_t* new_seq_lens, float* new_weights, int64_t new_weight_len,
                                       int32_t* kept, int budget, int recent, int num_seqs, int num_kv_heads,
                                       int head_dim, int block_size, int64_t num_blocks, pkv_stream_t stream) {
    if (num_seqs < 0) return fail(PKV_EINVAL, "num_seqs < 0");
    if (num_kv_heads <= 0) return fail(PKV_EINVAL, "num_kv_heads must be positive");
    if (head_dim != 64 && head_dim != 128) return fail(PKV_EUNSUPPORTED, "head_dim %d", head_dim);
    if (dtype_bytes(cache_dtype) == 0) return fail(PKV_EINVAL, "unknown dtype");
    if (block_size != 16 && block_size != 32) return fail(PKV_EUNSUPPORTED, "block_size %d", block_size);
    if (num_blocks <= 0 || num_blocks > 0x7fffffffLL) return fail(PKV_EINVAL, "num_blocks out of range");
    if (max_blocks_per_seq <= 0 || (int64_t)max_blocks_per_seq * block_size > 0x7fffffffLL ||
        new_max_blocks_per_seq <= 0 || (int64_t)new_max_blocks_per_seq * block_size > 0x7fffffffLL)
        return fail(PKV_EINVAL, "max_blocks_per_seq out of range");
    if (weight_len <= 0 || new_weight_len <= 0) return fail(PKV_EINVAL, "weight lengths must be positive");
    if (budget <= 0 || recent < 0 || recent > budget) return fail(PKV_EINVAL, "budget > 0 and 0 <= recent <= budget");
    if (num_seqs == 0) return PKV_OK;
    if (!key_cache || !value_cache || !block_tables || !seq_lens || !weights || !new_block_tables || !new_seq_lens ||
        !new_weights || !kept)
        return fail(PKV_EINVAL, "null pointer");
    if (!aligned16(key_cache) || !aligned16(value_cache)) return fail(PKV_EINVAL, "caches must be 16-byte aligned");
    if (new_weights == weights) return fail(PKV_EINVAL, "new_weights must not be weights");
    const int64_t rows = (int64_t)num_seqs * num_kv_heads;
    // destination blocks a sequence can have: as many as its new table and its tokens give
    const int64_t nblk = std::min<int64_t>(std::min<int64_t>(((int64_t)budget + block_size - 1) / block_size,
                                                             new_max_blocks_per_seq), max_blocks_per_seq);
    if (rows > 0x7fffffffLL || num_seqs * nblk > 0x7fffffffLL) return fail(PKV_EUNSUPPORTED, "too many rows");
    int* err = device_error_word();
    if (!err) return fail(PKV_ECUDA, "device error word unavailable");
    EvictParams p{};
    p.kc = static_cast<uint8_t*>(key_cache);
    p.vc = static_cast<uint8_t*>(value_cache);
    p.tables = block_tables; p.new_tables = new_block_tables; p.seq_lens = seq_lens; p.weights = weights;
    p.new_lens = new_seq_lens; p.new_weights = new_weights; p.kept = kept; p.err = err;
    p.weight_len = weight_len; p.new_weight_len = new_weight_len; p.num_blocks = num_blocks;
    p.num_seqs = num_seqs; p.hkv = num_kv_heads; p.mbps = max_blocks_per_seq; p.new_mbps = new_max_blocks_per_seq;
    p.bs = block_size; p.budget = budget; p.recent = recent; p.row_bytes = head_dim * dtype_bytes(cache_dtype);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    evict_select_kernel<<<(unsigned)rows, kSelThreads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "evict select launch: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_seqs * nblk));
    cfg.blockDim = dim3(kGatThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_gather_kernel, p, (int)nblk);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "evict gather launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}
