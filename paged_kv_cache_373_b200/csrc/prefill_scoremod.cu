// prefill_scoremod.cu -- pkv_paged_prefill_scoremod: chunked-prefill attention
// over the paged cache with modified scores.  A row at position p attends
//   t < prefix  or  (t <= p and t > p - window),
// with scores x = scale q.k, capped (cap tanh(x / cap)) and biased
// (- slope |p - t|).
//
// Unit: (sequence, kv head, 128 query rows), a row being a (chunk token, q head
// of the kv head's group) pair; a CTA takes two adjacent units of one (sequence,
// kv head), which read the same K/V tiles of 64 tokens:
//   - warps 0-3 and 4-7: the units' softmax, one thread per row, so that a row's
//     maximum and sum need no exchange: the 64 scores of a tile come from tensor
//     memory in one load, are capped, biased and masked in registers, exponentiated
//     against a reference maximum (by pairs, fp32x2), and P goes back over the scores
//     (bf16 as hi + lo parts: 32 + 32 columns, exactly the 64 of S), where the P V
//     product reads it as its A operand.  Every unit has two S buffers, so the scores
//     of the next tile are ready when a tile's P is done.  O stays in tensor memory and
//     is rescaled only when a row's maximum passes its reference by 2^8;
//   - warp 8 owns tensor memory (per unit two S of 64 and an O of
//     head_dim columns) and issues, per tile, O_0 += P_0 V, S_0'' = Q_0 K''^T, O_1 += P_1 V,
//     S_1'' = Q_1 K''^T (the tile after the next).  Products issued by one thread run in
//     order, so S'' may overwrite the P that the product before it reads;
//   - warp 9 copies the K and the V tiles (4-stage rings) with TMA through the block
//     table, a lane per box; warp 10 turns the copies' mbarriers into a counter, which
//     warp 8 reads together with the softmax warps', and completes the V tile that the
//     tokens end in with zeros.
// A pair's tiles are those that hold its prefix and then those from its earliest
// row's window on; the tiles between (tile kt of the walk is tile kt of the sequence
// up to the prefix's last, kt + gap after it) are left out.  A block of a walked tile
// that none of the pair's rows attends is copied from past the pool's end, which TMA
// fills with zeros: its table entry is not looked at.
// A unit without a partner (the odd one of a sequence; every unit where there are SMs for
// all) splits its tiles instead: group 0 takes the even tiles,
// group 1 the odd ones, and group 0 merges the two partial results at the end.
// Every hand-off is an mbarrier or a counter and every wait is bounded, as in prefill.cu.
//
// Measured (8192 rows of 16 / 8 heads of 128, bf16, scores capped; the last chunk of
// 2048 rows of 32 / 8 heads at 6100 with a window of 1024 and a prefix of 200): 160 us,
// 660 TFLOP/s of the algorithm's operations (P's lo part adds half as many again), and
// 66 to 73 us, replayed from a graph over the same inputs (called on changing ones 184 to 188
// and 74); one prompt of 8192 rows of 32 / 8 heads, capped, 800 TFLOP/s.  The plain prefill kernel's
// structure with these scores (two threads per row, one S buffer) took 294 and 123 us.
// What it took: 64-token tiles with two S buffers per unit and a cheaper cap, 284 -> 224
// and 159 -> 99; the issuing warp run uniformly with an elected lane (one lane's branch
// made every descriptor a vector register that the instruction had to fetch: 75 cycles a
// product), 3750 -> 2700 cycles per pair of tiles, and its waits as shared-memory
// counters -> 181 and 70; the cap, the maxima and the exponentials in one run without a
// branch -> 165 and 66; the pairs in the order of their lengths -> 160.  Bound now: the
// softmax warps, two per scheduler, whose instructions wait for each other's results
// (the schedulers issue in 47 % of the cycles, the tensor core is busy in 51 %, no pipe
// above 40 %).  Tried without gain: two threads per row (206 us: more warps, but 40 %
// more instructions), P beside S with S released early (190 us).  The 284 us are those of
// 128-token tiles in the kernel's first form; in the present one they are not measured.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "prefill.cuh"
#include "score_cap.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

using namespace tc;

constexpr int kRows = 128;          // query rows per unit (tensor-core M)
constexpr int kTok = 64;            // KV tokens per tile (N of S, K of P V)
constexpr int kStages = 4;          // ring depth: a stage holds V of tile j and K of tile j + ahead
constexpr int kSoftWarps = 8;       // 4 per unit: a thread per row
constexpr int kMmaWarp = 8, kWatchWarp = 10;  // (the copies: warp 9)
constexpr int kThreads = 11 * 32;
constexpr int kTmemCols = 512;      // S_X in columns 128 X + 64 (tile & 1).., O_X from 256 + 128 X

enum : int {
    kBarQ = 0,                       // q rows and the first `ahead` K tiles landed
    kBarFull = 1,                    // [stage] its V and K tile landed
    kBarEmpty = kBarFull + kStages,  // [stage] every product of the stage finished
    kBarStart = kBarEmpty + kStages, // the products of the first `ahead` K tiles finished
    kBarS = kBarStart + 1,           // [unit][buffer] S ready
    kBarO = kBarS + 4,               // [unit] P V of the tile before its last finished
    kBarEnd = kBarO + 2,             // [unit] its last P V finished
    kBarDrain = kBarEnd + 2,         // products drained
    kNumBars = kBarDrain + 1
};

// What the issuing warp waits for, as counters in shared memory that one load of
// the warp reads together (a wait on a finished mbarrier phase costs it 200 cycles,
// and it would need four per tile):
enum : int {
    kCntP = 0,  // [unit][softmax warp] tiles whose P is written
    kCntF = 8,  // stages filled (copied on from the mbarriers by kWatchWarp)
    kNumCnt = 32  // one per lane
};

struct PfMod {
    const float* slopes;         // [num_heads] or null
    const int32_t* prefix_lens;  // [num_seqs] or null
    float pre, inv_pre;          // scale / cap (0: no cap), cap / scale
    int window;                  // 0: no window
    int units;                   // per CTA: pairs (2), or every unit by itself (1)
};

// The tensor-core instructions of the issuing warp: every lane runs its loop, so
// that control flow is uniform and the descriptors stay in uniform registers,
// and the elected lane's predicate is on the instruction itself.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on));
}
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on));
}
__device__ __forceinline__ void commit(uint32_t on, uint32_t mbar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
                 ::"r"(mbar), "r"(on) : "memory");
}

__device__ __forceinline__ void publish(uint32_t addr, int n) {
    asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(addr), "r"(n) : "memory");
}

// The first n of a tile's 64 columns (none for n <= 0).
__device__ __forceinline__ uint64_t columns_below(int n) {
    return n <= 0 ? 0ull : n >= kTok ? ~0ull : (1ull << n) - 1;
}

struct Unit {
    int tok0, ntok, pos0, kv_end, nkv;
};

template <typename T, int D>
struct Smem {
    static constexpr int kQ = kRows * D * 2;     // one unit's q rows
    static constexpr int kTile = kTok * D * 2;   // one K or V tile
    static constexpr int kParts = std::is_same<T, __nv_bfloat16>::value ? 2 : 1;  // P hi (+ lo)
    static constexpr int kData = 2 * kQ + 2 * kStages * kTile + 1024;             // + alignment
    // at least 120 KB, so one CTA (and its 512 tensor-memory columns) per SM
    static constexpr int kBytes = kData > 120 * 1024 ? kData : 120 * 1024;
};

// Barrier over both softmax groups that also ORs a flag across them.
__device__ __forceinline__ bool soft_sync_or(bool flag) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}\n"
                 : "=r"(r) : "r"((uint32_t)flag), "n"(kSoftWarps * 32) : "memory");
    return r != 0;
}

// Warp-collective, 2 to 32 sequences, one per lane: the u-th longest unit pair of all,
// as (sequence, pair, the sequence's units); sequence -1 past the last.
__device__ __forceinline__ int3 pair_by_length(const PrefillParams& p, int units, int64_t u) {
    const int lane = threadIdx.x & 31, g = p.g;
    int C = 0, L = 0;
    if (lane < p.num_seqs) {
        C = chunk_rows(p, lane);
        L = __ldg(p.seq_lens + lane);
        if (C < 0 && blockIdx.x == 0 && threadIdx.x < 32) raise_error(p.err, PKV_DEVERR_SEQ_LEN);
    }
    const int nrt = C > 0 ? (int)(((int64_t)C * g + kRows - 1) / kRows) : 0;
    const int npr = (nrt + units - 1) / units;
    // pair j ends about (top - j) pairs' tokens into the sequence (top >= npr)
    const int step = units * kRows / g;
    const int top = max((int)(((int64_t)max(L, 0) + step - 1) / step), npr);
    if (u >= (int64_t)__reduce_add_sync(kFull, (unsigned)npr)) return make_int3(-1, 0, 0);
    // the highest x that at least u + 1 pairs reach
    auto reach = [&](int x) { return __reduce_add_sync(kFull, (unsigned)min(max(top - x + 1, 0), npr)); };
    int lo = 1, hi = __reduce_max_sync(kFull, npr > 0 ? top : 1);
    while (lo < hi) {
        const int x = lo + (hi - lo + 1) / 2;
        if (reach(x) > u) lo = x;
        else hi = x - 1;
    }
    const int at = (int)u - (int)reach(lo + 1);  // among those that end there
    const unsigned same = __ballot_sync(kFull, top - lo >= 0 && top - lo < npr);
    const unsigned hit = __ballot_sync(kFull, (same >> lane & 1) && __popc(same & ((1u << lane) - 1)) == at);
    const int s = max(__ffs(hit) - 1, 0);
    return make_int3(s, __shfl_sync(kFull, top - lo, s), __shfl_sync(kFull, nrt, s));
}

template <typename T, int D, bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
pkv_prefill_scoremod_kernel(const PrefillParams p, const __grid_constant__ CUtensorMap tmap_q,
                            const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                            const PfMod md) {
    using SM = Smem<T, D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int CB = D / 64;  // 128-byte column blocks per row
    extern __shared__ uint8_t pf_raw[];
    uint8_t* sm = pf_raw + ((1024 - (smem_u32(pf_raw) & 1023)) & 1023);  // 1024-byte aligned operands
    uint8_t* qsm = sm;                        // [2 units]
    uint8_t* ksm = qsm + 2 * SM::kQ;          // [stage]
    uint8_t* vsm = ksm + kStages * SM::kTile; // [stage]
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ int counters[kNumCnt];
    __shared__ float xsum[kRows], xref[kRows];  // group 1's row sums and references (split unit)
    volatile int* abort = &abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto stg = [](int kt) { return kt % kStages; };
    auto pass = [](int kt) { return (uint32_t)((kt / kStages) & 1); };

    // ---- the unit pair: kv head from the block index, then pair u among all
    // sequences' pairs (found by every warp).  A sequence's row tiles pair from the
    // last: (n-1, n-2), (n-3, n-4), ... (or every unit stands for itself).  Of 2 to 32 sequences, one per lane, the pairs
    // are taken in the order of their lengths, so that the grid's last CTAs are short
    // (the 8192 rows above: 160 us, by sequence 166); else sequence by sequence.
    const int kh = (int)(blockIdx.x % p.num_kv_heads);
    const int64_t u = blockIdx.x / p.num_kv_heads;
    int s = -1, jp = 0, nrt_s = 0;
    if (p.num_seqs > 1 && p.num_seqs <= 32) {
        const int3 at = pair_by_length(p, md.units, u);
        s = at.x;
        jp = at.y;
        nrt_s = at.z;
    } else {
        int64_t base = 0;
        // (block 0 goes through all of them, for its check)
        for (int s0 = 0; s0 < p.num_seqs && (s < 0 || blockIdx.x == 0); s0 += 32) {
            const int si = s0 + lane;
            int nrt = 0;
            if (si < p.num_seqs) {
                const int C = chunk_rows(p, si);
                if (C < 0 && blockIdx.x == 0 && warp == 0) raise_error(p.err, PKV_DEVERR_SEQ_LEN);
                nrt = C > 0 ? (int)(((int64_t)C * p.g + kRows - 1) / kRows) : 0;
            }
            const int npr = (nrt + md.units - 1) / md.units;
            int incl = npr;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += y;
            }
            const int64_t lo = base + incl - npr;
            const unsigned hit = __ballot_sync(kFull, npr > 0 && u >= lo && u < lo + npr);
            if (hit) {
                const int src = __ffs(hit) - 1;
                s = s0 + src;
                const int64_t l0 = __shfl_sync(kFull, lo, src);
                nrt_s = __shfl_sync(kFull, nrt, src);
                jp = (int)(u - l0);  // a sequence's heaviest pair first
            }
            base += __shfl_sync(kFull, incl, 31);
        }
    }
    if (s < 0) return;  // past the last pair
    const int q0 = __ldg(p.qstart + s), C = chunk_rows(p, s);
    const int L = __ldg(p.seq_lens + s);
    if (L < C || L > p.mbps * p.bs) {
        if (tid == 0) raise_error(p.err, PKV_DEVERR_SEQ_LEN);
        return;
    }
    const int pre = md.prefix_lens ? min(max(__ldg(md.prefix_lens + s), 0), L) : 0;
    const int window = md.window;
    const int tpu = kRows / p.g;  // chunk tokens per unit (g divides 16)
    const int j0 = nrt_s - 1 - md.units * jp, j1 = md.units == 2 ? j0 - 1 : -1;
    const int nunits = j1 >= 0 ? 2 : 1;
    auto make_unit = [&](int j) {
        Unit w;
        w.tok0 = j * tpu;
        w.ntok = min(tpu, C - w.tok0);
        w.pos0 = L - C + w.tok0;
        w.kv_end = max(w.pos0 + w.ntok, pre);
        w.nkv = (w.kv_end + kTok - 1) / kTok;
        return w;
    };
    Unit U0 = make_unit(j0);                 // the later rows: the longer K/V range
    Unit U1 = make_unit(j1 >= 0 ? j1 : j0);  // (the same when nunits == 1)
    // the walk's tiles: those of the prefix, then those from the earliest row's
    // window on.  Every unit has a row whose window starts at or after `first`
    // and ends before kv_end, so it keeps a tile past the gap.
    const int first = window > 0 ? max(U1.pos0 - window + 1, 0) : 0;
    const int gap = max(first / kTok - (pre + kTok - 1) / kTok, 0);
    U0.nkv -= gap;
    U1.nkv -= gap;
    const int nkv = U0.nkv;
    // With a bias the walk goes backwards, from the tiles at the rows' own positions: the
    // biased scores are highest there, so a row's reference stands from the start (8192
    // rows of 32 / 8 heads: 590 us; forwards it rises with nearly every tile, 1146 us).
    // Unit 1 then walks unit 0's tiles, at most two of which hold none of its tokens.
    constexpr bool kBack = kBias;
    if constexpr (kBack) U1.nkv = nkv;
    auto tile_token = [&](int kt) {
        const int k = kBack ? nkv - 1 - kt : kt;
        return (k * kTok < pre ? k : k + gap) * kTok;
    };
    // a unit alone splits its K/V tiles between the two groups (even / odd
    // tiles), whose partial results are merged at the end
    const bool split = nunits == 1;
    // S of a tile is issued two tiles of its unit ahead of its P V
    const int ahead = split ? 4 : 2;
    auto kstg = [&](int kt) { return (kt + kStages - ahead) % kStages; };  // ring slot of a K tile
    const bool need_fix = (U0.kv_end % kTok) != 0;  // V rows past the end must read as zeros

    // ---- tensor memory, barriers
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
    }
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), 1);
        for (int i = 0; i < kNumCnt; ++i) counters[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        abort_flag = 0;
    }
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = tmem_base;

    if (warp < kSoftWarps) {
        // ================= softmax group X: unit X (or, for a unit alone, its
        // tiles of parity X), a thread per row
        const int X = warp >> 2;
        const Unit U = X && !split ? U1 : U0;
        const int kt0 = split ? X : 0, kstep = split ? 2 : 1;  // this group's tiles
        const int ntiles = split ? (nkv - X + 1) / 2 : U.nkv;
        const int row = (warp & 3) * 32 + lane;
        const int pos = (row / p.g < U.ntok) ? U.pos0 + row / p.g : -1;
        const int last = U.pos0 + U.ntok - 1;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_addr + X * 128;
        const uint32_t tO = tmem + lane_addr + 256 + X * 128;
        const CapCoef cap = cap_coef(kCap ? md.pre : 1.f, kCap ? md.inv_pre : 1.f);
        const float sl2 = p.scale_log2;
        const float emul = kBias ? 1.f : sl2;  // without a bias the scale is applied in the exponent
        const float slope2 = kBias ? __ldg(md.slopes + (int64_t)kh * p.g + row % p.g) * 1.4426950408889634f : 0.f;
        float mref = -INFINITY, l = 0.f;  // reference maximum (log2 domain) and sum of the row
        bool failed = false;
#pragma unroll 1
        for (int i = 0; i < ntiles; ++i) {
            const int tt = tile_token(kt0 + i * kstep), buf = i & 1;
            const uint32_t tSb = tS + buf * kTok;
            bool ok = mbar_wait(bar(kBarS + 2 * X + buf), (i >> 1) & 1, abort, p.wait_ns);
            ok = __all_sync(kFull, ok);
            if (!ok) {
                failed = true;
                break;
            }
            tc_after_sync();
            // Most tiles: every column attended, no row's maximum far above its
            // reference and no score near the cap.  P is made on that assumption in one
            // straight run, which the compiler can interleave, and stored over the scores
            // only if it held for every row; otherwise the scores are read again below.
            // (Rows past the unit's end may hold anything.)
            const bool later = tt + kTok - 1 > U.pos0;  // a token past the first row
            const bool edge = (later || (window > 0 && tt <= last - window)) && tt + kTok > pre;
            bool done = false;
            // (the run's bias is for t <= p; walking back, a row may not have met its tokens yet)
            if (!edge && i > 0 && !(kBias && (later || __any_sync(kFull, mref == -INFINITY && pos >= 0)))) {
                float sc[kTok];
                tc_ld64(tSb, sc);
                const F2 sl = f2(sl2, sl2), minus1 = f2(-1.f, -1.f), one = f2(1.f, 1.f), s2 = f2(slope2, slope2);
                const float base = kBias ? -slope2 * (float)(pos - tt) - mref : -mref;
                const F2 base2 = f2(base, base);
                F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
                float big[2] = {0.f, 0.f}, top[2] = {-INFINITY, -INFINITY};
                uint32_t h[kTok / 2], lo[kTok / 2];
#pragma unroll
                for (int e = 0; e < kTok / 2; ++e) {
                    F2 v = f2(sc[2 * e], sc[2 * e + 1]);
                    if constexpr (kCap) {  // as cap_pairs
                        big[e & 1] = fmaxf(big[e & 1], fmaxf(fabsf(sc[2 * e]), fabsf(sc[2 * e + 1])));
                        const F2 z = f2_mul(v, v);
                        v = f2_mul(v, f2_fma(z, f2_fma(z, f2_fma(z, cap.c3, cap.c2), cap.c1), one));
                    }
                    const F2 bias = kBias ? f2_fma(s2, f2(2.f * e, 2.f * e + 1.f), base2) : base2;
                    const float2 x = f2_get(f2_fma(v, sl, bias));
                    top[e & 1] = fmaxf(top[e & 1], fmaxf(x.x, x.y));
                    const float a = ex2(x.x), b = ex2(x.y);
                    const F2 ab = f2(a, b);
                    sum[e & 1] = f2_add(sum[e & 1], ab);
                    // P in two bf16 parts, 16 bits; f16 keeps 11 in one, which next to the
                    // output's own 11 raises its error by 15 % (0.00020 -> 0.00023 of its size)
                    // and a second part would cost half as many products again
                    h[e] = pack2<kBf16>(a, b);
                    if constexpr (kBf16) {
                        const float2 hf = unpack2<true>(h[e]);
                        const float2 r = f2_get(f2_fma(f2(hf.x, hf.y), minus1, ab));
                        lo[e] = pack2<true>(r.x, r.y);
                    }
                }
                bool bad = !(fmaxf(top[0], top[1]) <= 8.f) || mref == -INFINITY;
                if constexpr (kCap) bad = bad || !(fmaxf(big[0], big[1]) < cap.lim);
                if (!__any_sync(kFull, bad && pos >= 0)) {
#pragma unroll
                    for (int c = 0; c < kTok / 2; c += 16) {
                        tc_st16u(tSb + c, h + c);
                        if constexpr (kBf16) tc_st16u(tSb + kTok / 2 + c, lo + c);
                    }
                    const float2 t = f2_get(f2_add(sum[0], sum[1]));
                    l += t.x + t.y;
                    done = true;
                }
            }
            if (!done) {
            float sc[kTok];
            tc_ld64(tSb, sc);
            if constexpr (kCap) cap_pairs(sc, cap);
            if constexpr (kBias) {
                const float d0 = (float)(pos - tt);
#pragma unroll
                for (int c = 0; c < kTok; ++c) sc[c] = fmaf(sc[c], sl2, -slope2 * fabsf(d0 - (float)c));
            }
            // tiles with a token past the first row, or at or before the last row's window
            if (edge) {
                const uint64_t vis = columns_below(pre - tt) |
                                     (columns_below(pos - tt + 1) & ~(window > 0 ? columns_below(pos - window + 1 - tt) : 0ull));
                const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    sc[c] = v0 & (1u << c) ? sc[c] : -INFINITY;
                    sc[32 + c] = v1 & (1u << c) ? sc[32 + c] : -INFINITY;
                }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kTok; c += 2) m4[(c >> 1) & 3] = fmaxf(m4[(c >> 1) & 3], fmaxf(sc[c], sc[c + 1]));
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * emul;
            const bool grow = mx > mref + 8.f;  // also the first finite maximum
            float alpha = 1.f;
            if (grow) {
                alpha = ex2(mref - mx);  // 0 while nothing was attended
                l *= alpha;
                mref = mx;
            }
            if (i > 0 && __any_sync(kFull, grow)) {  // rescale O, once the previous tile's product is in it
                // (S of the next tile was issued after it; the last tile has a barrier for it)
                ok = i + 1 < ntiles ? mbar_wait(bar(kBarS + 2 * X + (buf ^ 1)), ((i + 1) >> 1) & 1, abort, p.wait_ns)
                                    : mbar_wait(bar(kBarO + X), 0, abort, p.wait_ns);
                ok = __all_sync(kFull, ok);
                if (!ok) {
                    failed = true;
                    break;
                }
                tc_after_sync();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                    float v[16];
                    tc_ld16(tO + c0, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] *= alpha;
                    tc_st16(tO + c0, v);
                }
            }
            const float ref = mref == -INFINITY ? 0.f : mref;
            const F2 em2 = f2(emul, emul), nref2 = f2(-ref, -ref), minus1 = f2(-1.f, -1.f);
            F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
            for (int c0 = 0; c0 < kTok; c0 += 32) {  // P over the scores, two tokens per 32-bit column
                uint32_t h[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 x = f2_get(f2_fma(f2(sc[c0 + 2 * e], sc[c0 + 2 * e + 1]), em2, nref2));
                    const float a = ex2(x.x), b = ex2(x.y);
                    const F2 ab = f2(a, b);
                    sum[e & 1] = f2_add(sum[e & 1], ab);
                    h[e] = pack2<kBf16>(a, b);
                    if constexpr (kBf16) {
                        const float2 hf = unpack2<true>(h[e]);
                        const float2 r = f2_get(f2_fma(f2(hf.x, hf.y), minus1, ab));
                        lo[e] = pack2<true>(r.x, r.y);
                    }
                }
                tc_st16u(tSb + c0 / 2, h);
                if constexpr (kBf16) tc_st16u(tSb + kTok / 2 + c0 / 2, lo);
            }
            const float2 s2 = f2_get(f2_add(sum[0], sum[1]));
            l += s2.x + s2.y;
            }
            tc_wait_st();
            tc_before_sync();
            __syncwarp();
            if (lane == 0) publish(smem_u32(&counters[kCntP + warp]), i + 1);
        }
        // ---- the last P V, then normalise (a split unit also merges group 1's
        // partial result) and store
        bool ok = !failed && (ntiles == 0 || mbar_wait(bar(kBarEnd + X), 0, abort, p.wait_ns));
        if (split && X == 0 && nkv > 1) ok = ok && mbar_wait(bar(kBarEnd + 1), 0, abort, p.wait_ns);  // read in the merge
        ok = __all_sync(kFull, ok);
        bool merge = false;
        if (split) {
            if (X == 1) {
                xsum[row] = l;
                xref[row] = mref;
            }
            ok = !soft_sync_or(!ok);
            merge = nkv > 1;
        }
        if (ok && !(split && X == 1)) {
            tc_after_sync();
            float lt = l, a0 = 1.f, a1 = 0.f;
            if (merge) {
                const float m1 = xref[row], m = fmaxf(mref, m1);
                a0 = mref == -INFINITY ? 0.f : ex2(mref - m);
                a1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
                lt = a0 * lt + a1 * xsum[row];
            }
            const float inv = lt > 0.f ? 1.f / lt : 0.f;
            a0 *= inv;
            a1 *= inv;
            T* out = static_cast<T*>(p.out) +
                     ((int64_t)(q0 + U.tok0 + row / p.g) * p.num_heads + (int64_t)kh * p.g + row % p.g) * D;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
                float v[16];
                tc_ld16(tO + c0, v);  // every lane loads (warp-collective); only real rows store
                if (merge) {
                    float v1[16];
                    tc_ld16(tO + 128 + c0, v1);  // group 1's O
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = a0 * v[e] + a1 * v1[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] *= a0;
                }
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = pack2<kBf16>(v[2 * e], v[2 * e + 1]);
                if (pos >= 0) {
                    *reinterpret_cast<uint4*>(out + c0) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(out + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        }
    } else if (warp == kMmaWarp) {
        // ================= tensor-core issue
        {
            const uint32_t on = elect_one();
            const uint32_t id_s = tc_idesc<kBf16>(kRows, kTok, 0);
            const uint32_t id_o = tc_idesc<kBf16>(kRows, D, 1);
            const uint64_t dq0 = tc_desc(smem_u32(qsm), 16, 1024);
            const uint64_t dq1 = tc_desc(smem_u32(qsm + (split ? 0 : SM::kQ)), 16, 1024);
            const uint64_t dk0 = tc_desc(smem_u32(ksm), 16, 1024);
            const uint64_t dv0 = tc_desc(smem_u32(vsm), kTok * 128, 1024);
            // S_X = Q_X K^T into buffer b (a split unit: both groups read q slot 0)
            auto issue_s = [&](int X, int b, int st) {
                const uint64_t qd = X ? dq1 : dq0;
                const uint64_t kd = desc_add(dk0, (uint32_t)(st * (SM::kTile >> 4)));
                const uint32_t d = tmem + X * 128 + b * kTok;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(on, d, desc_add(qd, ((kk >> 2) * kRows * 128 + (kk & 3) * 32) >> 4),
                           desc_add(kd, ((kk >> 2) * kTok * 128 + (kk & 3) * 32) >> 4), id_s, kk > 0);
                commit(on, bar(kBarS + 2 * X + b));
            };
            // O_X (+)= P_X V (hi, then lo; P over S_X in buffer b)
            auto issue_pv = [&](int X, int b, int st, bool acc) {
                const uint64_t vd = desc_add(dv0, (uint32_t)(st * (SM::kTile >> 4)));
                const uint32_t d = tmem + 256 + X * 128, a = tmem + X * 128 + b * kTok;
#pragma unroll
                for (int part = 0; part < SM::kParts; ++part)
#pragma unroll
                    for (int kk = 0; kk < kTok / 16; ++kk)
                        mma_ts(on, d, a + part * (kTok / 2) + kk * 8, desc_add(vd, (kk * 2048) >> 4), id_o,
                               (acc || part > 0 || kk > 0) ? 1u : 0u);
            };
            // The counters are read ahead (look), before products whose issue takes
            // longer than the load; reached waits until every lane's counter is at the
            // lane's target (bounded as mbar_wait).
            const uint32_t cnt = smem_u32(&counters[lane]);
            int seen = 0;
            auto look = [&]() {
                asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(seen) : "r"(cnt) : "memory");
            };
            auto reached = [&](int target) {
                uint64_t t0 = 0;
                for (uint32_t it = 1;; ++it) {
                    if (__all_sync(kFull, seen >= target)) {
                        __syncwarp();  // what any lane acquired, the issuing lane has
                        tc_after_sync();
                        return true;
                    }
                    if ((it & 255) == 0) {
                        bool stop = *abort != 0;
                        const uint64_t now = global_ns();
                        if (t0 == 0) t0 = now;
                        else if (now - t0 > p.wait_ns) stop = true;
                        if (__any_sync(kFull, stop)) {
                            if (lane == 0) *abort = 1;
                            return false;
                        }
                    }
                    look();
                }
            };
            // this lane's target: n tiles' P of unit X, f stages
            auto target = [&](int X, int n, int f) {
                return lane < kCntF ? (lane >> 2 == X ? n : -1) : lane == kCntF ? f : -1;
            };
            bool ok = __all_sync(kFull, mbar_wait(bar(kBarQ), 0, abort, p.wait_ns)) != 0;
            if (ok) {
                tc_after_sync();
                const int n = min(ahead, nkv);
#pragma unroll 1
                for (int kt = 0; kt < n; ++kt) {
                    if (split) {
                        issue_s(kt & 1, kt >> 1, kstg(kt));
                    } else {
                        issue_s(0, kt, kstg(kt));
                        if (kt < U1.nkv) issue_s(1, kt, kstg(kt));
                    }
                }
                commit(on, bar(kBarStart));
                look();
            }
            if (!split) {
                // paired units: every tile serves both; per tile kt
                // O_0 += P_0 V, S_0 of tile kt + 2, O_1 += P_1 V, S_1 of tile kt + 2
#pragma unroll 1
                for (int kt = 0; ok && kt < nkv; ++kt) {
                    const int st = stg(kt), b = kt & 1;
                    const bool n0 = kt + 2 < nkv, a1 = kt < U1.nkv, a1n = kt + 2 < U1.nkv;
                    ok = reached(target(0, kt + 1, kt + 1));
                    if (!ok) break;
                    issue_pv(0, b, st, kt > 0);
                    if (kt == nkv - 2) commit(on, bar(kBarO));
                    if (kt == nkv - 1) commit(on, bar(kBarEnd));
                    look();
                    if (n0) issue_s(0, b, st);
                    if (a1) {
                        ok = reached(target(1, kt + 1, 0));
                        if (!ok) break;
                        issue_pv(1, b, st, kt > 0);
                        if (kt == U1.nkv - 2) commit(on, bar(kBarO + 1));
                        if (kt == U1.nkv - 1) commit(on, bar(kBarEnd + 1));
                        look();
                        if (a1n) issue_s(1, b, st);
                    }
                    commit(on, bar(kBarEmpty + st));
                }
            } else {
                // a split unit: group X = kt & 1 takes tile kt into its buffer (kt >> 1) & 1
#pragma unroll 1
                for (int kt = 0; ok && kt < nkv; ++kt) {
                    const int X = kt & 1, b = (kt >> 1) & 1, st = stg(kt);
                    ok = reached(target(X, (kt >> 1) + 1, kt + 1));
                    if (!ok) break;
                    issue_pv(X, b, st, kt > 1);
                    if (kt + 2 < nkv && kt + 4 >= nkv) commit(on, bar(kBarO + X));
                    if (kt + 2 >= nkv) commit(on, bar(kBarEnd + X));
                    look();
                    if (kt + 4 < nkv) issue_s(X, b, st);
                    commit(on, bar(kBarEmpty + st));
                }
            }
            commit(on, bar(kBarDrain));  // every product issued has finished before tensor memory is freed
            mbar_wait(bar(kBarDrain), 0, nullptr, p.wait_ns);
        }
        __syncwarp();
    } else if (warp == kWatchWarp) {
        // ================= the copies' mbarriers, passed on as a counter; the last token's
        // V tile is completed with zeros first
        bool ok = true;
#pragma unroll 1
        for (int j = 0; ok && j < nkv; ++j) {
            ok = mbar_wait(bar(kBarFull + stg(j)), pass(j), abort, p.wait_ns);
            ok = __all_sync(kFull, ok);
            if (ok && need_fix && j == (kBack ? 0 : nkv - 1)) {  // V rows at and past the unit's end
                const int r0 = U0.kv_end - tile_token(j);
                uint8_t* vt = vsm + stg(j) * SM::kTile;
                constexpr int CH = D / 8;  // 16-byte chunks per row
                for (int i = lane; i < (kTok - r0) * CH; i += 32)
                    *reinterpret_cast<uint4*>(vt + tc_off(r0 + i / CH, i % CH, kTok)) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
            }
            if (ok && lane == 0) publish(smem_u32(&counters[kCntF]), j + 1);
        }
    } else {
        // ================= TMA copies: the q rows, then stage by stage V of tile j
        // (lanes 0-7) and K of tile j + ahead (lanes 8-15), a lane per 64-element box
        const bool is_k = (lane >> 3) & 1;
        const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
        const int jb = (lane & 7) / CB, cb = (lane & 7) % CB;  // this lane's block of a tile and column block
        const int32_t* trow = p.tables + (int64_t)s * p.mbps;
        const int lg_bs = p.bs == 16 ? 4 : 5;
        const int kt_end = p.stop_tile < 0 ? nkv : min(nkv, p.stop_tile);
        const uint32_t box_bytes = (uint32_t)p.bs * 128;
        // whether this lane has a box of tile kt (of K or V, as is_k says)
        auto has_box = [&](int kt, bool kind) {
            return kind && kt < nkv && jb < (kTok >> lg_bs) && tile_token(kt) + (jb << lg_bs) < U0.kv_end;
        };
        auto copy = [&](int kt, int b) {
            const int t = tile_token(kt) + (jb << lg_bs);
            int phys = (int)p.num_blocks;  // a block that no row attends: zeros from past the pool
            if (t < pre || t + p.bs > first) {
                phys = __ldg(trow + (t >> lg_bs));
                if (phys < 0 || phys >= p.num_blocks) {
                    raise_error(p.err, PKV_DEVERR_BLOCK_ID);
                    phys = 0;
                }
            }
            uint8_t* tile = is_k ? ksm + kstg(kt) * SM::kTile : vsm + stg(kt) * SM::kTile;
            tma_load3(smem_u32(tile + cb * kTok * 128 + jb * p.bs * 128), map, cb * 64, kh, phys * p.bs, bar(b));
        };
        // the q rows and the first K tiles, announced together
        const int nfirst = min(ahead, kt_end);
        uint32_t bytes = (uint32_t)(nunits * SM::kQ);
        for (int kt = 0; kt < nfirst; ++kt)
            bytes += __popc(__ballot_sync(kFull, has_box(kt, lane >= 8 && lane < 16))) * box_bytes;
        if (lane == 0) mbar_expect_tx(bar(kBarQ), bytes);
        __syncwarp();
        if (lane < nunits * CB) {
            const int X = lane / CB, qc = lane % CB;
            tma_load3(smem_u32(qsm + X * SM::kQ + qc * kRows * 128), &tmap_q, qc * 64, kh * p.g,
                      q0 + (X ? U1.tok0 : U0.tok0), bar(kBarQ));
        }
        for (int kt = 0; kt < nfirst; ++kt)
            if (has_box(kt, lane >= 8 && lane < 16)) copy(kt, kBarQ);
        bool ok = true;
        int issued = 0;  // stages
#pragma unroll 1
        for (int j = 0; j < kt_end; ++j) {
            // the first stages whose K tile goes where one of the first was; then
            // the stages used before
            if (j == kStages - ahead) ok = mbar_wait(bar(kBarStart), 0, abort, p.wait_ns);
            if (j >= kStages) ok = ok && mbar_wait(bar(kBarEmpty + stg(j)), pass(j - kStages), abort, p.wait_ns);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            const int kt = is_k ? j + ahead : j;
            const bool on = has_box(kt, lane < 16);
            const uint32_t n = __popc(__ballot_sync(kFull, on));
            if (lane == 0) mbar_expect_tx(bar(kBarFull + stg(j)), n * box_bytes);
            __syncwarp();
            if (on) copy(kt, kBarFull + stg(j));
            ++issued;
        }
        if (kt_end < nkv) ok = false;  // (timeout test) the other roles wait for the missing tiles
        if (!ok) {  // let the copies in flight land before the CTA ends
            mbar_wait(bar(kBarQ), 0, nullptr, p.wait_ns);
            for (int j = max(issued - kStages, 0); j < issued; ++j)
                mbar_wait(bar(kBarFull + stg(j)), pass(j), nullptr, p.wait_ns);
        }
    }

    tc_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
    if (tid == 0 && abort_flag) raise_error(p.err, PKV_DEVERR_TIMEOUT);
}

template <typename T, int D, bool kCap, bool kBias>
pkv_status launch(const PrefillParams& p, const PfMod& md, const void* query, const void* kc, const void* vc,
                  int64_t num_tokens, int64_t grid, cudaStream_t st) {
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kSmem = Smem<T, D>::kBytes;
    static_assert(kSmem <= 227 * 1024 - 4 * 1024, "shared memory");
    CUtensorMap tq, tk, tv;
    pkv_status r = encode_map(&tq, kBf16, query, D, p.num_heads, num_tokens, p.g, kRows / p.g);
    if (r == PKV_OK) r = encode_map(&tk, kBf16, kc, D, p.num_kv_heads, p.num_blocks * p.bs, 1, p.bs);
    if (r == PKV_OK) r = encode_map(&tv, kBf16, vc, D, p.num_kv_heads, p.num_blocks * p.bs, 1, p.bs);
    if (r != PKV_OK) return r;
    static std::atomic<unsigned long long> configured{0};  // bit per device (< 64)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(PKV_ECUDA, "cudaGetDevice");
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(pkv_prefill_scoremod_kernel<T, D, kCap, kBias>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return fail(PKV_ECUDA, "prefill smem opt-in: %s", cudaGetErrorString(e));
        configured.fetch_or(bit);
    }
    pkv_prefill_scoremod_kernel<T, D, kCap, kBias><<<(unsigned)grid, kThreads, kSmem, st>>>(p, tq, tk, tv, md);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "prefill launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

template <typename T, int D>
pkv_status dispatch(const PrefillParams& p, const PfMod& md, const void* query, const void* kc, const void* vc,
                    int64_t num_tokens, int64_t grid, cudaStream_t st) {
    if (md.slopes)
        return md.pre > 0.f ? launch<T, D, true, true>(p, md, query, kc, vc, num_tokens, grid, st)
                            : launch<T, D, false, true>(p, md, query, kc, vc, num_tokens, grid, st);
    return md.pre > 0.f ? launch<T, D, true, false>(p, md, query, kc, vc, num_tokens, grid, st)
                        : launch<T, D, false, false>(p, md, query, kc, vc, num_tokens, grid, st);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_paged_prefill_scoremod(
    void* out, const void* query, pkv_dtype q_dtype, const void* key_cache, const void* value_cache,
    pkv_dtype cache_dtype, const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
    const int32_t* query_start, int num_seqs, int64_t num_query_tokens, int num_heads, int num_kv_heads,
    int head_dim, int block_size, int64_t num_blocks, float scale, float softcap, int window,
    const float* alibi_slopes, const int32_t* prefix_lens, pkv_stream_t stream) {
    PrefillParams p;
    int64_t grid = 0;
    pkv_status st = prefill_prepare(&p, &grid, out, query, q_dtype, key_cache, value_cache, cache_dtype, block_tables,
                                    max_blocks_per_seq, seq_lens, query_start, num_seqs, num_query_tokens, num_heads,
                                    num_kv_heads, head_dim, block_size, num_blocks, scale);
    if (st != PKV_OK) return st;
    PfMod md{alibi_slopes, prefix_lens, 0.f, 0.f, window, 2};
    float cap2 = 0.f, inv_cap2 = 0.f;
    st = score_cap(softcap, &cap2, &inv_cap2);
    if (st != PKV_OK) return st;
    if (window < 0) return fail(PKV_EINVAL, "window < 0");
    if ((int64_t)max_blocks_per_seq * block_size > 0x40000000LL)  // positions and windows add up in 32 bits
        return fail(PKV_EUNSUPPORTED, "table rows of more than 2^30 tokens");
    if (window >= max_blocks_per_seq * block_size) md.window = 0;  // hides nothing
    if (grid == 0) return PKV_OK;
    md.pre = p.scale_log2 * inv_cap2;
    md.inv_pre = 1.f / md.pre;
    if (softcap > 0.f && !(md.pre >= 0x1p-126f && md.pre <= 0x1p126f)) {
        // scale / cap next to or past the ends of fp32.  Below 2^-126 the cap changes no
        // product q.k under 2^114 in its 24 bits, and 2^-126 gives the same; above 2^126
        // tanh is 1 for every product but 0, whichever of the two multiplies it, and
        // what is left is the cap itself.
        const double r = (double)scale / (double)softcap;
        md.pre = r < 1.0 ? 0x1p-126f : 0x1p126f;
        md.inv_pre = r < 1.0 ? 0x1p126f : (float)(1.0 / r);
    }
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int64_t T = num_query_tokens;
    // Where every unit can have an SM of its own (sum_s ceil(C_s g / 128) <= T g / 128 + S),
    // units stand alone and split their tiles: half the tiles one after the other.
    // Chunks of 273, 542, 14 and 606 tokens of 8 / 4 heads of 64: 13.6 us, in pairs 19.6;
    // 900 tokens at 3000: 48.0, in pairs 85.7.  With more units than SMs the pairs, which
    // read a K/V tile once for both, mostly win (200 units of 8 / 4 heads of 128 at 6000:
    // 199 us against 244).
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return fail(PKV_ECUDA, "cannot size the grid");
    const int64_t alone = (T * p.g / kRows + num_seqs) * num_kv_heads;
    if (alone <= sms) {
        md.units = 1;
        grid = alone;
    }
    if (cache_dtype == PKV_F16)
        return head_dim == 64 ? dispatch<__half, 64>(p, md, query, key_cache, value_cache, T, grid, cs)
                              : dispatch<__half, 128>(p, md, query, key_cache, value_cache, T, grid, cs);
    return head_dim == 64 ? dispatch<__nv_bfloat16, 64>(p, md, query, key_cache, value_cache, T, grid, cs)
                          : dispatch<__nv_bfloat16, 128>(p, md, query, key_cache, value_cache, T, grid, cs);
}
