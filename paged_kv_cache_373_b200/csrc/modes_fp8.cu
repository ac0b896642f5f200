// Decode variants for FP8 E4M3 caches: modified scores, and scores kept for the
// accumulated attention weights.  Tile shapes as in attn_fp8.cu.
#include "attn_launch.cuh"

namespace pkv {
namespace {
template <class QT, class Arg>
pkv_status by_block(const DecodeLaunchArgs& a, const Arg& x, cudaStream_t s) {
    if (a.params->block_size % 32 == 0) return launch_decode_k<Cfg<uint8_t, QT, 128, Path::kFp8, 8, 2, 32>>(a, x, s);
    return launch_decode_k<Cfg<uint8_t, QT, 128, Path::kFp8, 12, 3>>(a, x, s);
}
template <class Arg>
pkv_status dispatch(const DecodeLaunchArgs& a, const Arg& x, bool q_bf16, cudaStream_t s) {
    return q_bf16 ? by_block<__nv_bfloat16>(a, x, s) : by_block<__half>(a, x, s);
}
}  // namespace

pkv_status launch_mod_fp8(const DecodeLaunchArgs& a, const ModArg& m, bool q_bf16, cudaStream_t s) {
    return dispatch(a, m, q_bf16, s);
}
pkv_status launch_scores_fp8(const DecodeLaunchArgs& a, const WeightsArg& w, bool q_bf16, cudaStream_t s) {
    return dispatch(a, WeightsArg2{w}, q_bf16, s);
}
}  // namespace pkv
