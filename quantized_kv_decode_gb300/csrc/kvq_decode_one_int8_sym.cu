// Decode of many short contexts, a warp each: symmetric INT8 caches.
#include "kvq_decode_fast.cuh"

namespace kvq {

template <int D, int NG>
static cudaError_t by_gp(const DecodeParams& p, int gp, cudaStream_t s, bool* handled, int* occ) {
  *handled = true;
  switch (gp) {
    case 1: return fast::launch_one_inst<8, D, NG, 1, true>(p, s, occ);
    case 2: return fast::launch_one_inst<8, D, NG, 2, true>(p, s, occ);
    case 4: if constexpr (NG * 4 <= 16) return fast::launch_one_inst<8, D, NG, 4, true>(p, s, occ);
            break;
    case 8: if constexpr (NG * 8 <= 16) return fast::launch_one_inst<8, D, NG, 8, true>(p, s, occ);
            break;
  }
  *handled = false;
  return cudaSuccess;
}

cudaError_t launch_decode_one_int8_sym(const DecodeParams& p, int gp, cudaStream_t s, bool* handled, int* occ) {
  *handled = false;
  const int D = p.geom.D, NG = p.geom.ngroups;
  if (D == 128 && NG == 2) return by_gp<128, 2>(p, gp, s, handled, occ);
  if (D == 128 && NG == 4) return by_gp<128, 4>(p, gp, s, handled, occ);
  if (D == 128 && NG == 8) return by_gp<128, 8>(p, gp, s, handled, occ);
  if (D == 64 && NG == 2) return by_gp<64, 2>(p, gp, s, handled, occ);
  if (D == 64 && NG == 4) return by_gp<64, 4>(p, gp, s, handled, occ);
  return cudaSuccess;
}

}  // namespace kvq
