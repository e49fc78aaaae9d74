// Decode of many short contexts, a warp each: INT2 caches.
#include "kvq_decode_fast.cuh"

namespace kvq {

template <int NG, bool SYM>
static cudaError_t by_gp(const DecodeParams& p, int gp, cudaStream_t s, bool* handled, int* occ) {
  *handled = true;
  switch (gp) {
    case 1: return fast::launch_one_inst<2, 128, NG, 1, SYM>(p, s, occ);
    case 2: if constexpr (NG * 2 <= 8) return fast::launch_one_inst<2, 128, NG, 2, SYM>(p, s, occ);
            break;
    case 4: if constexpr (NG == 2) return fast::launch_one_inst<2, 128, NG, 4, SYM>(p, s, occ);
            break;
    case 8: if constexpr (NG == 2) return fast::launch_one_inst<2, 128, NG, 8, SYM>(p, s, occ);
            break;
  }
  *handled = false;
  return cudaSuccess;
}

cudaError_t launch_decode_one_int2(const DecodeParams& p, int gp, cudaStream_t s, bool* handled, int* occ) {
  *handled = false;
  const int NG = p.geom.ngroups;
  if (p.geom.D != 128) return cudaSuccess;
  if (p.geom.sym) {
    if (NG == 2) return by_gp<2, true>(p, gp, s, handled, occ);
    if (NG == 4) return by_gp<4, true>(p, gp, s, handled, occ);
    if (NG == 8) return by_gp<8, true>(p, gp, s, handled, occ);
  } else {
    if (NG == 2) return by_gp<2, false>(p, gp, s, handled, occ);
    if (NG == 4) return by_gp<4, false>(p, gp, s, handled, occ);
    if (NG == 8) return by_gp<8, false>(p, gp, s, handled, occ);
  }
  return cudaSuccess;
}

}  // namespace kvq
