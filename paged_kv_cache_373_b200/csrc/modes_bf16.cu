// Decode variants for bf16 caches: modified scores, and scores kept for the
// accumulated attention weights.  Tile shapes as in attn_bf16.cu.
#include "attn_launch.cuh"

namespace pkv {
namespace {
template <class Arg>
pkv_status dispatch(const DecodeLaunchArgs& a, const Arg& x, int head_dim, cudaStream_t s) {
    if (head_dim == 64)
        return launch_decode_k<Cfg<__nv_bfloat16, __nv_bfloat16, 64, Path::kMma16, kWarps16, 4>>(a, x, s);
    return launch_decode_k<Cfg<__nv_bfloat16, __nv_bfloat16, 128, Path::kMma16, kWarps16, 2>>(a, x, s);
}
}  // namespace

pkv_status launch_mod_bf16(const DecodeLaunchArgs& a, const ModArg& m, int head_dim, cudaStream_t s) {
    return dispatch(a, m, head_dim, s);
}
pkv_status launch_scores_bf16(const DecodeLaunchArgs& a, const WeightsArg& w, int head_dim, cudaStream_t s) {
    return dispatch(a, w, head_dim, s);
}
}  // namespace pkv
