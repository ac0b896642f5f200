// evict.cu -- pkv_evict_tokens: cache eviction by accumulated attention weight.
// Per (sequence, kv head) with more tokens than the budget, the last `recent`
// tokens and the heaviest of the others stay, in ascending order, and their K/V
// rows move to the first `budget` slots of a new block table.
//
// Two kernels.
//   select: one CTA per (sequence, kv head) finds the budget's threshold on the
//     weights' bits, then numbers the kept tokens in order by ballots and one sum over
//     the warps.  Integer work only, so the result does not depend on any order.  A row
//     of up to kBatch weights is loaded once, stays in registers and is searched two bits
//     at a time, by the whole CTA until few keys share the prefix and then by one warp; a
//     longer one is read again for each of three histograms (11 + 11 + 10 bits; on a row
//     that fits the registers they took 2.4 us more) and once more for the numbering.
//     Bound: issue slots, 1500 instructions a warp, and the passes' barriers.
//   gather: one CTA per destination block copies its rows, 16 bytes per thread and
//     access.  The blocks that hold recent tokens alone need nothing of the selection
//     and are copied beside it.  Bound: memory -- every kept row is read and written
//     once; a row is at least one 64-byte run.
// 32 sequences of 1000 to 8192 tokens, 8 kv heads of 128 x 16 bits, budget 2048, recent
// 512: 64.5 us, 5580 GB/s.  Without the early blocks and the one warp it was 77.5 us.
// One sequence of 8192 tokens, 8 kv heads: 18 us; of 20000 40.7 us.  1024 threads with 31
// keys each take 29.6 us there, but 71.5 for the 32 sequences above.
// The source and the destination are different blocks, so nothing is moved onto
// rows still to be read, blocks shared with other sequences stay as they are, and
// the copy needs no order.
#include <algorithm>
#include <type_traits>

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
constexpr int kList = 512;                          // keys that one warp searches alone
static_assert(kList <= kBins, "they lie in the histogram's memory");

// Order-preserving map of a weight to an unsigned key; NaN is the lowest, -0 is +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The weight of a key, but for the two keys that stand for several bit patterns, NaN's
// and zero's.
__device__ __forceinline__ float key_weight(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ bool key_is_exact(uint32_t key) { return key != 0u && key != 0x80000000u; }

// How many of the warp's keys (n per lane, at most 16) are not below each of three
// candidates, 10 bits each: two bits of a threshold for one reduction.
template <int N>
__device__ __forceinline__ uint32_t count3(const uint32_t (&key)[N], int n, uint32_t c1, uint32_t c2, uint32_t c3) {
    static_assert(N * 32 < 1024, "10 bits");
    uint32_t a = 0, b = 0, c = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i >= n) break;
        a += key[i] >= c1 ? 1u : 0u;
        b += key[i] >= c2 ? 1u << 10 : 0u;
        c += key[i] >= c3 ? 1u << 20 : 0u;
    }
    return __reduce_add_sync(kFull, a + b + c);
}

// The candidates of the next step below `bit` (the last step has one bit, and two that no
// key reaches), and the step's result: the highest of them that at least `want` keys
// reach becomes the prefix.  lo, hi: keys not below the prefix, and above those that
// share it.
struct Step {
    int sh;
    uint32_t c1, c2, c3;
    __device__ __forceinline__ Step(uint32_t prefix, int bit) {
        sh = bit > 0 ? bit - 1 : 0;
        c1 = prefix | (1u << sh);
        c2 = bit > 0 ? prefix | (2u << sh) : ~0u;
        c3 = bit > 0 ? prefix | (3u << sh) : ~0u;
    }
    __device__ __forceinline__ void take(int n1, int n2, int n3, int want, int& bit, uint32_t& prefix, int& lo, int& hi) {
        if (n3 >= want) prefix = c3, lo = n3;
        else if (n2 >= want) prefix = c2, lo = n2, hi = n3;
        else if (n1 >= want) prefix = c1, lo = n1, hi = bit > 0 ? n2 : hi;
        else hi = n1;
        bit = sh - 1;
    }
};

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

__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads)
evict_select_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int hist[kBins];
    __shared__ int wsum[kSelWarps];
    __shared__ int count[2][kSelWarps], kept_of[2][kSelWarps];
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
    const int nw_len = (int)min(p.new_weight_len, (int64_t)p.budget);
    auto keep = [&](int j, int t, float weight) {
        if (j < p.budget) kept[j] = t;
        if (j < nw_len) nw[j] = weight;
    };
    if (L <= p.budget) {  // everything stays where it is
        for (int j = tid; j < p.budget; j += kSelThreads) {
            if (j < L) keep(j, j, w[j]);
            else kept[j] = -1;
        }
        return;
    }
    const int m = L - p.recent;       // tokens to choose from
    const int c = p.budget - p.recent;  // of which c stay (0 <= c < m)
    auto keep_recent = [&] {
        for (int t = m + tid; t < L; t += kSelThreads) keep(c + t - m, t, w[t]);
    };
    if (c == 0) {
        keep_recent();
        return;
    }

    // the weights of a batch, all loads in flight; a row that fits one batch is
    // loaded once and stays in registers through the passes.  A warp holds `per` runs
    // of 32 tokens, one behind the other, so that the order of the kept tokens
    // needs no sums across warps but one.
    const bool one = m <= kBatch;
    const int per = one ? (m + kSelThreads - 1) / kSelThreads : kKeys;
    const int t0 = warp * per * 32 + lane;  // the thread's first token, from the batch's
    uint32_t key[kKeys];
    auto load = [&](int base, auto meanwhile) {
        float x[kKeys];
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (i >= per) break;  // (the same for every thread, here and below)
            const int t = base + t0 + 32 * i;
            x[i] = t < m ? w[t] : 0.f;
        }
        meanwhile();
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (i >= per) break;
            key[i] = base + t0 + 32 * i < m ? weight_key(x[i]) : 0u;  // 0: below every candidate
        }
    };
    auto nothing = [] {};
    if (one) load(0, keep_recent);
    else keep_recent();

    // ---- the c-th largest key.  A row in registers: by two bits from the highest bit in
    // which its keys differ, by counting the keys not below a candidate, until exactly c
    // are; once kList keys or fewer share the prefix those go on alone, in one
    // warp.  A longer row: three digits by histograms, one reading of the row each.
    uint32_t prefix = 0;
    int left = c;  // rank still to find among the keys that share the prefix
    if (one) {
        uint32_t all = ~0u, any = 0u;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (i >= per) break;
            any |= key[i];
            if (t0 + 32 * i < m) all &= key[i];
        }
        all = __reduce_and_sync(kFull, all);
        any = __reduce_or_sync(kFull, any);
        if (lane == 0) {
            count[0][warp] = (int)all;
            count[1][warp] = (int)any;
        }
        if (tid == 0) sh_left = 0;
        __syncthreads();
        all = __reduce_and_sync(kFull, lane < kSelWarps ? (uint32_t)count[0][lane] : ~0u);
        any = __reduce_or_sync(kFull, lane < kSelWarps ? (uint32_t)count[1][lane] : 0u);
        __syncthreads();
        int bit = 31 - __clz(all ^ any);  // -1: all keys are equal
        prefix = bit < 0 ? all : all & ~((2u << bit) - 1);
        int lo = m, hi = 0;  // keys not below the prefix; keys above those that share it
        bool exact = false;
        for (int buf = 0; bit >= 0 && !exact && lo - hi > kList; buf ^= 1) {
            Step step(prefix, bit);
            const uint32_t mine = count3(key, per, step.c1, step.c2, step.c3);
            if (lane == 0) count[buf][warp] = (int)mine;
            __syncthreads();
            const uint32_t v = lane < kSelWarps ? (uint32_t)count[buf][lane] : 0u;
            step.take((int)__reduce_add_sync(kFull, v & 1023u), (int)__reduce_add_sync(kFull, v >> 10 & 1023u),
                      (int)__reduce_add_sync(kFull, v >> 20), c, bit, prefix, lo, hi);
            exact = lo == c;
        }
        if (bit >= 0 && !exact) {
            const uint32_t low = (2u << bit) - 1;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (i >= per) break;
                const bool in = t0 + 32 * i < m && (key[i] ^ prefix) <= low;
                const unsigned who = __ballot_sync(kFull, in);
                if (who == 0) continue;
                int at = 0;
                if (lane == 0) at = atomicAdd(&sh_left, __popc(who));  // (their order is of no matter)
                at = __shfl_sync(kFull, at, 0) + __popc(who & ((1u << lane) - 1));
                if (in && at < kBins) hist[at] = (int)key[i];
            }
            __syncthreads();
            if (warp == 0) {
                constexpr int kOwn = kList / 32;
                const int own = (lo - hi + 31) / 32;  // keys a lane has (<= kOwn)
                uint32_t mine[kOwn];
#pragma unroll
                for (int i = 0; i < kOwn; ++i) mine[i] = 32 * i + lane < lo - hi ? (uint32_t)hist[32 * i + lane] : 0u;
                left = c - hi;
                int in = lo - hi, above = 0;  // of these keys
                while (bit >= 0 && in != left) {
                    Step step(prefix, bit);
                    const uint32_t v = count3(mine, own, step.c1, step.c2, step.c3);
                    step.take((int)(v & 1023u), (int)(v >> 10 & 1023u), (int)(v >> 20), left, bit, prefix, in, above);
                }
                if (in == left) prefix -= 1, left = 0;  // the keys not below the prefix
                else left -= above;
                if (lane == 0) {
                    sh_digit = prefix;
                    sh_left = left;
                }
            }
            __syncthreads();
            prefix = sh_digit;
            left = sh_left;
        } else if (exact) {
            prefix -= 1;  // the c keys not below the prefix
            left = 0;
        } else {
            left = c - hi;  // all keys that share the prefix are equal
        }
    } else {
        constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t mask = d == 0 ? 0u : 0xffffffffu << (kShift[d] + kBits[d]);
            for (int base = 0; base < m; base += kBatch) {
                load(base, nothing);
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    const uint32_t k = key[i];
                    if (base + t0 + 32 * i < m && (k & mask) == prefix)
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

    // ---- number the kept tokens in order: the ballots of a warp's runs, one sum over
    // the warps, and the totals of the batches before.  `ties` false: left is 0, no
    // token is kept for its equal key, which halves the work.
    const unsigned below = (1u << lane) - 1;
    auto number = [&](auto ties) {
        constexpr bool kTies = decltype(ties)::value;
        int gt0 = 0, eq0 = 0;
        for (int base = 0; base < m; base += kBatch) {
            if (!one) load(base, nothing);
            auto equal = [&](int i) {
                return kTies ? __ballot_sync(kFull, base + t0 + 32 * i < m && key[i] == prefix) : 0u;
            };
            auto above = [&](int i) { return __ballot_sync(kFull, key[i] > prefix); };  // (a key past the row is 0)
            int ng = 0, ne = 0;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (i >= per) break;
                ng += __popc(above(i));
                ne += __popc(equal(i));
            }
            if (lane == 0) {
                kept_of[0][warp] = ng;
                kept_of[1][warp] = ne;
            }
            __syncthreads();
            const int vg = lane < kSelWarps ? kept_of[0][lane] : 0, ve = kTies && lane < kSelWarps ? kept_of[1][lane] : 0;
            int g = gt0 + __reduce_add_sync(kFull, lane < warp ? vg : 0);
            int e = kTies ? eq0 + (int)__reduce_add_sync(kFull, lane < warp ? ve : 0) : 0;
            // The weights go out from their keys: reading each again would wait for the
            // stores before it (the compiler cannot know that they are apart), 74 us
            // against 66 in the case above.  The kept zeros and NaN are read afterwards.
            uint32_t again = 0;
            const int g_first = g, e_first = e;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                if (i >= per) break;
                const unsigned ba = above(i), be = equal(i);
                const bool is_eq = be >> lane & 1;
                const int rank = e + __popc(be & below);
                if (key[i] > prefix || (is_eq && rank < left)) {
                    const int j = g + __popc(ba & below) + min(rank, left);
                    keep(j, base + t0 + 32 * i, key_weight(key[i]));
                    if (!key_is_exact(key[i])) again |= 1u << i;
                }
                g += __popc(ba);
                e += __popc(be);
            }
            if (__any_sync(kFull, again != 0)) {
                int g2 = g_first, e2 = e_first;
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    if (i >= per) break;
                    const unsigned ba = above(i), be = equal(i);
                    const int j = g2 + __popc(ba & below) + min(e2 + __popc(be & below), left);
                    if ((again >> i & 1) && j < nw_len) nw[j] = w[base + t0 + 32 * i];
                    g2 += __popc(ba);
                    e2 += __popc(be);
                }
            }
            if (one) break;
            gt0 += __reduce_add_sync(kFull, vg);
            if (kTies) eq0 += __reduce_add_sync(kFull, ve);
            __syncthreads();
        }
    };
    if (left == 0) number(std::false_type{});
    else number(std::true_type{});
}

// One row per thread and turn: two in flight cost 3 us more in the case above, 256
// threads 1 us more.
constexpr int kGatThreads = 512;

// CTA: part `part` of destination block b of sequence s (one part, unless the blocks are
// so few that their rows' dependent loads would be waited for in turn: one sequence of 6206
// tokens to 1000, 8 kv heads, 15.8 us in 8 parts, 18.8 in one).  kLanes threads hold a row, 16 bytes
// each; the CTA's rows (slot, head) are walked in the destination's order, which is
// one contiguous run, so no index needs a division.
template <int kLanes>
__global__ void __launch_bounds__(kGatThreads)
evict_gather_kernel(const EvictParams p, int nblk, int parts, int lg_bs) {
    constexpr int kStep = kGatThreads / kLanes;  // rows the CTA copies side by side
    constexpr int kRowBytes = kLanes * 16;
    // the sequences' last blocks first
    const int part = (int)(blockIdx.x % parts), unit = (int)(blockIdx.x / parts);
    const int s = unit % p.num_seqs, b = nblk - 1 - unit / p.num_seqs;
    bool bad;
    const int L = evict_len(p, s, &bad);
    // A block of recent tokens alone depends on nothing of the selection and goes on
    // beside it; the grid's last CTA always waits, so that the grid ends after it.
    const bool early = b * p.bs >= p.budget - p.recent;
    if (early && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool on = L > p.budget;
    const int dst = on ? __ldg(p.new_tables + (int64_t)s * p.new_mbps + b) : 0;
    const int c = threadIdx.x % kLanes, r0 = part * kStep + threadIdx.x / kLanes, step = parts * kStep;
    int slot = r0 / p.hkv, h = r0 - slot * p.hkv;
    const int dslot = step / p.hkv, dh = step - dslot * p.hkv;
    if (!early) asm volatile("griddepcontrol.wait;" ::: "memory");
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
        const int t = early ? L - p.budget + b * p.bs + slot : kept[(int64_t)h * p.budget + slot];
        if ((unsigned)t < (unsigned)L) {
            const int src = __ldg(table + (t >> lg_bs));
            if (src < 0 || src >= p.num_blocks) {
                if (c == 0) raise_error(p.err, PKV_DEVERR_BLOCK_ID);
            } else {
                const int64_t from = ((((int64_t)src << lg_bs) + (t & (p.bs - 1))) * p.hkv + h) * kRowBytes + 16 * c;
                const uint4 k = *reinterpret_cast<const uint4*>(p.kc + from);
                const uint4 v = *reinterpret_cast<const uint4*>(p.vc + from);
                *reinterpret_cast<uint4*>(p.kc + to) = k;
                *reinterpret_cast<uint4*>(p.vc + to) = v;
            }
        }
        slot += dslot;
        h += dh;
        if (h >= p.hkv) { h -= p.hkv; ++slot; }
        to += (int64_t)step * kRowBytes;
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
    // What the call writes lies apart from all that it reads and from what else it writes: other
    // CTAs of a sequence still read its length, table and weights when its first results are stored.
    const Span reads[] = {{"seq_lens", seq_lens, 4.0 * num_seqs},
                          {"weights", weights, 4.0 * rows * weight_len},
                          {"block_tables", block_tables, 4.0 * num_seqs * max_blocks_per_seq},
                          {"new_block_tables", new_block_tables, 4.0 * num_seqs * new_max_blocks_per_seq}};
    const Span writes[] = {{"new_seq_lens", new_seq_lens, 4.0 * num_seqs},
                           {"new_weights", new_weights, 4.0 * rows * new_weight_len},
                           {"kept", kept, 4.0 * rows * budget}};
    for (int i = 0; i < 3; ++i) {
        for (const Span& r : reads)
            if (overlap(writes[i], r)) return fail(PKV_EINVAL, "%s overlaps %s", writes[i].name, r.name);
        for (int j = 0; j < i; ++j)
            if (overlap(writes[i], writes[j])) return fail(PKV_EINVAL, "%s overlaps %s", writes[i].name, writes[j].name);
    }
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
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t steps = ((int64_t)block_size * num_kv_heads * p.row_bytes / 16 + kGatThreads - 1) / kGatThreads;
    const int parts = (int)std::max<int64_t>(1, std::min(steps, 4 * (int64_t)sms / (num_seqs * nblk)));
    cfg.gridDim = dim3((unsigned)(num_seqs * nblk * parts));
    cfg.blockDim = dim3(kGatThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int lg_bs = block_size == 16 ? 4 : 5;
    switch (p.row_bytes / 16) {
    case 4: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<4>, p, (int)nblk, parts, lg_bs); break;
    case 8: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<8>, p, (int)nblk, parts, lg_bs); break;
    case 16: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<16>, p, (int)nblk, parts, lg_bs); break;
    default: e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<32>, p, (int)nblk, parts, lg_bs); break;
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "evict gather launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}
