// Rotary positions: rotation of q and k (kvq_rope_apply), and the rotation
// fused into the quantizing append (kvq_rope_append).
#include "kvq_rope_kernels.cuh"

namespace kvq {

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  const long long total = (long long)p.batch * p.num_new;
  if (total == 0 || p.Hq + p.Hk == 0) return cudaSuccess;
  if (rope_vec(p.rope)) {
    RopeAppendParams q{};
    q.r = p;
    return launch_warp<0, 0>(q, stream);
  }
  int tokens;
  dim3 grid;
  rope_grid(total, p.Hq + p.Hk, 1, &tokens, &grid);
  return launch2(rope_kernel<RopeParams>, grid, kThreads, turn_bytes(p.rope, tokens), stream, p, tokens);
}

cudaError_t launch_rope_append(const RopeAppendParams& p, cudaStream_t stream) { return launch_append_any(p, stream); }

}  // namespace kvq
