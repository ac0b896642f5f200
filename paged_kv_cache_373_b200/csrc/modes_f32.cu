// Decode variants for fp32 caches: modified scores, and scores kept for the
// accumulated attention weights.  Tile shapes as in attn_f32.cu.
#include "attn_launch.cuh"

namespace pkv {
namespace {
template <class Arg>
pkv_status dispatch(const DecodeLaunchArgs& a, const Arg& x, int head_dim, cudaStream_t s) {
    if (head_dim == 64) return launch_decode_k<Cfg<float, float, 64, Path::kF32, 8, 2>>(a, x, s);
    return launch_decode_k<Cfg<float, float, 128, Path::kF32, 4, 2>>(a, x, s);
}
}  // namespace

pkv_status launch_mod_f32(const DecodeLaunchArgs& a, const ModArg& m, int head_dim, cudaStream_t s) {
    return dispatch(a, m, head_dim, s);
}
pkv_status launch_scores_f32(const DecodeLaunchArgs& a, const WeightsArg& w, int head_dim, cudaStream_t s) {
    return dispatch(a, w, head_dim, s);
}
}  // namespace pkv
