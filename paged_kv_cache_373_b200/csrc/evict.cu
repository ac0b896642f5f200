// evict.cu -- pkv_evict_tokens: cache eviction by accumulated attention weight.
// Per (sequence, kv head) with more tokens than the budget, the last `recent`
// tokens and the heaviest of the others stay, in ascending order, and their K/V
// rows move to the first `budget` slots of a new block table.
//
// Two kernels.
//   select: one CTA per (sequence, kv head) finds the budget's threshold on the
//     weights' bits, then numbers the kept tokens in order by ballots and one scan.
//     Integer work only, so the result does not depend on any order.  A row of up to
//     kBatch weights is loaded once, stays in registers and is searched bit by bit
//     (at most 33 counts); a longer one is read again for each of three histograms
//     (11 + 11 + 10 bits) and once more for the numbering.  Bound: the latency of
//     its barriers.
//   gather: one CTA per destination block copies its rows, 16 bytes per thread and
//     access, K and V of four rows in flight together.  Bound: memory -- every kept row is read
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

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
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

__global__ void __launch_bounds__(kSelThreads, 2)
evict_select_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int hist[kBins];
    __shared__ int wsum[kSelWarps];
    __shared__ int run_gt[kRuns], run_eq[kRuns];
    __shared__ int count[2][kSelWarps];
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
        if (j >= p.budget) return;
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
            if (base + i * kSelThreads >= m) break;  // (the same for every thread, here and below)
            const int t = base + i * kSelThreads + tid;
            x[i] = t < m ? w[t] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (base + i * kSelThreads >= m) break;
            key[i] = base + i * kSelThreads + tid < m ? weight_key(x[i]) : 0u;  // 0: below every candidate
        }
    };
    const bool one = m <= kBatch;
    if (one) load(0);

    // ---- the c-th largest key.  A row in registers: bit by bit from the top, by
    // counting the keys not below a candidate; done early when exactly c are.  A
    // longer row: three digits by histograms, one reading of the row each.
    uint32_t prefix = 0;
    int left = c;  // rank still to find among the keys that share the prefix
    if (one) {
        auto at_least = [&](uint32_t cand, int buf) {  // cand > 0: keys past the row are 0
            int n = 0;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (i * kSelThreads >= m) break;
                n += key[i] >= cand;
            }
            n = __reduce_add_sync(kFull, n);
            if (lane == 0) count[buf][warp] = n;
            __syncthreads();
            return __reduce_add_sync(kFull, lane < kSelWarps ? count[buf][lane] : 0);
        };
        bool exact = false;
        for (int b = 31; b >= 0 && !exact; --b) {
            const uint32_t cand = prefix | (1u << b);
            const int n = at_least(cand, b & 1);
            if (n >= c) prefix = cand;
            exact = n == c;
        }
        if (exact) {
            prefix -= 1;  // the c keys not below the candidate
            left = 0;
        } else {
            left = c - at_least(prefix + 1, 1);
        }
    } else {
        constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t mask = d == 0 ? 0u : 0xffffffffu << (kShift[d] + kBits[d]);
            for (int base = 0; base < m; base += kBatch) {
                load(base);
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    if (base + i * kSelThreads >= m) break;
                    const uint32_t k = key[i];
                    if (base + i * kSelThreads + tid < m && (k & mask) == prefix)
                        atomicAdd(&hist[(k >> kShift[d]) & ((1u << kBits[d]) - 1)], 1);
                }
            }
            __syncthreads();
            // thread i holds kPerThread bins, counted from the top down
            constexpr int kPerThread = kBins / kSelThreads;
            int own = 0;
#pragma unroll
            for (int q = 0; q < kPerThread; ++q) own += hist[kBins - 1 - kPerThread * tid - q];
            int incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += y;
            }
            if (lane == 31) wsum[warp] = incl;
            __syncthreads();
            int before = incl - own;  // keys in higher bins
            for (int q = 0; q < warp; ++q) before += wsum[q];
            if (left > before && left <= before + own) {
                int q = 0;
                while (true) {
                    const int n = hist[kBins - 1 - kPerThread * tid - q];
                    if (left <= before + n) break;
                    before += n;
                    ++q;
                }
                sh_digit = (uint32_t)(kBins - 1 - kPerThread * tid - q);
                sh_left = left - before;
            }
            __syncthreads();
            prefix |= sh_digit << kShift[d];
            left = sh_left;
        }
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
            unsigned bg = 0, be = 0;
            if (base + i * kSelThreads < m) {
                const bool in = base + i * kSelThreads + tid < m;
                bg = __ballot_sync(kFull, in && key[i] > prefix);
                be = __ballot_sync(kFull, in && key[i] == prefix);
            }
            if (lane == 0) {
                run_gt[i * kSelWarps + warp] = __popc(bg);
                run_eq[i * kSelWarps + warp] = __popc(be);
            }
        }
        __syncthreads();
        if (warp < 2) {  // exclusive scan of kRuns counts, kOwn per lane; warp 0: gt, warp 1: eq
            constexpr int kOwn = kRuns / 32;
            static_assert(kOwn * 32 == kRuns, "every run has its lane");
            int* run = (warp ? run_eq : run_gt) + lane * kOwn;
            int v[kOwn], sum = 0;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                v[i] = run[i];
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
            for (int i = 0; i < kOwn; ++i) {
                run[i] = x;
                x += v[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (base + i * kSelThreads >= m) break;
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
constexpr int kGatRows = 2;  // rows a thread has in flight

// CTA: destination block b of sequence s.  kLanes threads hold a row, 16 bytes
// each; the CTA's rows (slot, head) are walked in the destination's order, which is
// one contiguous run, so no index needs a division.
template <int kLanes>
__global__ void __launch_bounds__(kGatThreads)
evict_gather_kernel(const EvictParams p, int nblk, int lg_bs) {
    constexpr int kStep = kGatThreads / kLanes;  // rows the CTA copies side by side
    constexpr int kRowBytes = kLanes * 16;
    const int s = (int)(blockIdx.x / nblk), b = (int)(blockIdx.x % nblk);
    bool bad;
    const int L = evict_len(p, s, &bad);
    const bool on = L > p.budget;
    const int dst = on ? __ldg(p.new_tables + (int64_t)s * p.new_mbps + b) : 0;
    const int c = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
    int slot = r0 / p.hkv, h = r0 - slot * p.hkv;
    const int dslot = kStep / p.hkv, dh = kStep - dslot * p.hkv;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!on) return;
    if (dst < 0 || dst >= p.num_blocks) {
        if (threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const int slots = min(p.bs, p.budget - b * p.bs);
    const int32_t* table = p.tables + (int64_t)s * p.mbps;
    const int32_t* kept = p.kept + (int64_t)s * p.hkv * p.budget + b * p.bs;
    int64_t to = ((int64_t)dst * p.bs * p.hkv + r0) * kRowBytes + 16 * c;
    while (slot < slots) {
        int t[kGatRows], hh[kGatRows];
        bool in[kGatRows];
#pragma unroll
        for (int i = 0; i < kGatRows; ++i) {
            in[i] = slot < slots;
            hh[i] = h;
            t[i] = in[i] ? kept[(int64_t)h * p.budget + slot] : 0;
            if ((unsigned)t[i] >= (unsigned)L) { t[i] = 0; in[i] = false; }
            slot += dslot;
            h += dh;
            if (h >= p.hkv) { h -= p.hkv; ++slot; }
        }
        int src[kGatRows];
#pragma unroll
        for (int i = 0; i < kGatRows; ++i) src[i] = __ldg(table + (t[i] >> lg_bs));
        uint4 k[kGatRows], v[kGatRows];
#pragma unroll
        for (int i = 0; i < kGatRows; ++i) {
            if (in[i] && (src[i] < 0 || src[i] >= p.num_blocks)) {
                if (c == 0) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
                in[i] = false;
            }
            if (in[i]) {
                const int64_t from = ((((int64_t)src[i] << lg_bs) + (t[i] & (p.bs - 1))) * p.hkv + hh[i]) * kRowBytes + 16 * c;
                k[i] = *reinterpret_cast<const uint4*>(p.kc + from);
                v[i] = *reinterpret_cast<const uint4*>(p.vc + from);
            }
        }
#pragma unroll
        for (int i = 0; i < kGatRows; ++i) {
            if (in[i]) {
                *reinterpret_cast<uint4*>(p.kc + to) = k[i];
                *reinterpret_cast<uint4*>(p.vc + to) = v[i];
            }
            to += kStep * kRowBytes;
        }
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
    if ((int64_t)max_blocks_per_seq * block_size > 0x40000000LL)  // 32-bit token indexes with room for a batch
        return fail(PKV_EUNSUPPORTED, "table rows of more than 2^30 tokens");
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
    const int lg_bs = block_size == 16 ? 4 : 5;
    switch (p.row_bytes / 16) {
    case 4: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<4>, p, (int)nblk, lg_bs); break;
    case 8: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<8>, p, (int)nblk, lg_bs); break;
    case 16: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<16>, p, (int)nblk, lg_bs); break;
    default: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<32>, p, (int)nblk, lg_bs); break;
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "evict gather launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}
