// attn_launch.cuh -- launcher template shared by the per-variant
// translation units (attn_*.cu): opt the kernel into its shared-memory size
// once per device, launch the decode kernel (one warp = one worker) and the
// split-merge kernel (one warp per worker boundary).
#pragma once

#include <atomic>
#include <cstdio>

#include "paged_attention.cuh"
#include "pkv_internal.h"

namespace pkv {

// The decode grid with one of the two length-scan forms.
template <class C, class Arg, bool kWideScan>
pkv_status launch_decode_grid(const DecodeLaunchArgs& a, const Arg& sx, cudaStream_t st) {
    static std::atomic<unsigned long long> configured{0};  // bit per device (< 64)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(PKV_ECUDA, "cudaGetDevice");
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(pkv_decode_kernel<C, Arg, kWideScan>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   C::kSmemBytes);
        if (e != cudaSuccess) return fail(PKV_ECUDA, "smem opt-in: %s", cudaGetErrorString(e));
        configured.fetch_or(bit);
    }
    const DecodeParams& p = *a.params;
    cudaError_t e = cudaSuccess;
    if constexpr (Arg::kSuffix) {
        // the cascade suffix pass: a programmatic dependent of the prefix pass
        // (it may start on SMs the prefix pass leaves; see WaitPrimaryAtExit)
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)a.grid);
        cfg.blockDim = dim3(C::kWarps * 32);
        cfg.dynamicSmemBytes = C::kSmemBytes;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, pkv_decode_kernel<C, Arg, kWideScan>, p, sx);
    } else {
        pkv_decode_kernel<C, Arg, kWideScan><<<a.grid, C::kWarps * 32, C::kSmemBytes, st>>>(p, sx);
    }
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "decode launch: %s", cudaGetErrorString(e));
    return PKV_OK;
}

// CTAs of the weights pass: an item each (4 tokens per thread), at most
// kWeightCtas per CTA of the persistent grid.
inline int64_t weight_ctas(const DecodeParams& p, int grid, int threads) {
    const int64_t cap = (int64_t)p.max_blocks_per_seq * p.block_size;
    const int64_t items = (int64_t)p.num_seqs * p.num_kv_heads * ((cap + 4 * threads - 1) / (4 * threads));
    const int64_t most = (int64_t)kWeightCtas * grid;
    return items < most ? items : most;
}

template <class C, class Arg>
pkv_status launch_decode_k(const DecodeLaunchArgs& a, const Arg& sx, cudaStream_t st) {
    static_assert(C::kSmemBytes + sizeof(BlockScanSmem) <= 227 * 1024, "shared memory budget");
    const DecodeParams& p = *a.params;
    // the length scans: each warp alone while one round of a warp's scan
    // covers the batch, else once per CTA
    const pkv_status ds = p.num_seqs > 32 * kScanPerLane ? launch_decode_grid<C, Arg, true>(a, sx, st)
                                                          : launch_decode_grid<C, Arg, false>(a, sx, st);
    if (ds != PKV_OK) return ds;
    if (Arg::kSuffix && a.skip_merge) return PKV_OK;  // the cascade's finish pass merges the split units
    cudaError_t e = cudaSuccess;
    // the merge kernel is a programmatic dependent launch: its CTAs start
    // while the decode grid drains, locate their unit from the lengths (which
    // the decode kernel does not write) and wait for the decode grid's results
    // only before reading the workspace
    const int64_t workers = (int64_t)a.grid * C::kWarps;
    cudaLaunchConfig_t cfg = {};
    // one CTA per worker boundary (a warp per head row), or for batches
    // whose length scan takes more than two rounds of a warp, 8 boundaries
    // per CTA located by one CTA-wide scan
    const bool wide = p.num_seqs > 2 * 32 * kScanPerLane;
    if constexpr (Arg::kMod || Arg::kWeights) {
        // small batches of the variants: a CTA per unit (see pkv_merge_units_kernel)
        const int64_t units = (int64_t)p.num_seqs * p.num_kv_heads * p.nch;
        if (p.num_seqs <= 32 * kScanPerLane && units <= workers) {
            cudaLaunchAttribute pdl[1];
            pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            pdl[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.gridDim = dim3((unsigned)units);
            cfg.blockDim = dim3(kUnitWarps * 32);
            cfg.stream = st;
            cfg.attrs = pdl;
            cfg.numAttrs = 1;
            bool with_weights = false;
            if constexpr (Arg::kWeights) {
                // the weights pass in the same grid while its items are few (one
                // launch less: 1.4 us of 9.7 for 5 sequences of up to 777 tokens; for
                // 64 of up to 8192 tokens it took 8 us more, every CTA making its own
                // log sums)
                const int64_t ctas = weight_ctas(p, a.grid, kUnitWarps * 32);
                with_weights = ctas <= 2 * (int64_t)a.grid && p.g <= kWeightGroup;
                if (with_weights) {
                    cfg.gridDim = dim3((unsigned)(units + ctas));
                    e = cudaLaunchKernelEx(&cfg, pkv_merge_weights_kernel<typename C::q_t, C::D, C::kTT, Arg>, p, workers, sx);
                }
            }
            if (!with_weights)
                e = cudaLaunchKernelEx(&cfg, pkv_merge_units_kernel<typename C::q_t, C::D, C::kTT, Arg>, p, workers, sx);
            if (e == cudaSuccess) e = cudaGetLastError();
            if (e != cudaSuccess) return fail(PKV_ECUDA, "merge launch: %s", cudaGetErrorString(e));
            if constexpr (Arg::kWeights)
                if (!with_weights) return launch_weights_pass(p, sx, a.grid, st);
            return PKV_OK;
        }
    }
    cfg.gridDim = dim3((unsigned)(wide ? (workers + kMergeWarps - 1) / kMergeWarps : workers));
    cfg.blockDim = dim3(32 * (wide ? kMergeWarps : p.hpu));
    cfg.dynamicSmemBytes = 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (wide)
        e = cudaLaunchKernelEx(&cfg, pkv_merge_wide_kernel<typename C::q_t, C::D, C::kTT, Arg>, p, workers, sx);
    else
        e = cudaLaunchKernelEx(&cfg, pkv_merge_kernel<typename C::q_t, C::D, C::kTT, Arg>, p, workers, sx);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(PKV_ECUDA, "merge launch: %s", cudaGetErrorString(e));
    if constexpr (Arg::kWeights) return launch_weights_pass(p, sx, a.grid, st);
    return PKV_OK;
}

// Plain decode, or the cascade suffix pass when the call asks for it.
template <class C>
pkv_status launch_decode(const DecodeLaunchArgs& a, cudaStream_t st) {
    if (!a.suffix) return launch_decode_k<C>(a, SuffixArg<false>{}, st);
    return launch_decode_k<C>(a, SuffixArg<true>{a.seq_start, a.part_o, a.part_ml, a.prefix_eff, a.cta_ticket,
                                                 a.num_groups, a.prefix_units, a.prefix_tile}, st);
}

}  // namespace pkv
