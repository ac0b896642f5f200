// Decode variants for f16 caches: modified scores, and scores kept for the
// accumulated attention weights.  Tile shapes as in attn_f16.cu.
#include "attn_launch.cuh"

namespace pkv {
namespace {
template <class Arg>
pkv_status dispatch(const DecodeLaunchArgs& a, const Arg& x, int head_dim, cudaStream_t s) {
    if (head_dim == 64) return launch_decode_k<Cfg<__half, __half, 64, Path::kMma16, kWarps16, 4>>(a, x, s);
    return launch_decode_k<Cfg<__half, __half, 128, Path::kMma16, kWarps16, 2>>(a, x, s);
}
}  // namespace

pkv_status launch_mod_f16(const DecodeLaunchArgs& a, const ModArg& m, int head_dim, cudaStream_t s) {
    return dispatch(a, m, head_dim, s);
}
pkv_status launch_scores_f16(const DecodeLaunchArgs& a, const WeightsArg& w, int head_dim, cudaStream_t s) {
    return dispatch(a, WeightsArg2{w}, head_dim, s);
}
}  // namespace pkv
