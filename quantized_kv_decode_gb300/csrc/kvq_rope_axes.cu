// Rotary positions by several axes (kvq_rope_axes_apply, kvq_rope_axes_append):
// the kernels of kvq_rope_kernels.cuh with a position for each pair's axis.
#include "kvq_rope_kernels.cuh"

namespace kvq {

cudaError_t launch_rope_axes(const RopeAxesParams& p, cudaStream_t stream) {
  const long long total = (long long)p.r.batch * p.r.num_new;
  if (total == 0 || p.r.Hq + p.r.Hk == 0) return cudaSuccess;
  if (rope_vec(p.r.rope)) return launch_warp<0, 0>(p, stream);
  int tokens;
  dim3 grid;
  rope_grid(total, p.r.Hq + p.r.Hk, 1, &tokens, &grid);
  return launch2(rope_kernel<RopeAxesParams>, grid, kThreads, turn_bytes(p.r.rope, tokens), stream, p, tokens);
}

cudaError_t launch_rope_axes_append(const RopeAxesParams& p, cudaStream_t stream) {
  return launch_append_any(p, stream);
}

}  // namespace kvq
