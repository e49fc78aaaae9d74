// Cached rows back to fp16 (kvq_cache_read): one thread per 8 channels of a
// row, grid y = K / V.  Bound by memory: codes and headers in, fp16 rows out.
#include "kvq_load.cuh"

namespace kvq {
namespace {

template <int BITS>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheGeom& c = p.v.geom;
  const int which = p.out[0] ? blockIdx.y : 1;
  const int chunks = c.D / 8;
  const long long n = (long long)p.batch * p.num_rows * c.Hkv * chunks;
  const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= n) return;
  const int ch = (int)(u % chunks);
  long long r = u / chunks;
  const int kvh = (int)(r % c.Hkv);
  r /= c.Hkv;
  const int b = (int)(r / p.num_rows), t = (int)(r - (long long)b * p.num_rows);
  const int L = checked_len(c, p.seq_lens, b, -1);
  const int s0 = __ldg(p.start + b);
  uint32_t flags = 0;
  if (L < 0 || L > cache_capacity(c) || s0 < 0) {
    flags = KVQ_FLAG_SEQ_LEN;
  } else if ((long long)s0 + t < L) {
    const int pos = s0 + t;
    const long long row = view_row(c, b, kvh, L, pos);
    if (row < 0) {
      flags = KVQ_FLAG_BLOCK_TABLE;
    } else {
      const uint4 x = load8<BITS>(p.v, which, b, kvh, L, pos, row, ch);
      uint4* o = reinterpret_cast<uint4*>(p.out[which]) + u;
      if (KVQ_IN(c, which ? KVQ_ARRAY_V_NEW : KVQ_ARRAY_K_NEW, o, 16)) *o = x;
    }
  }
  if (flags && ch == 0 && p.status) atomicOr(p.status, flags);
}

}  // namespace

cudaError_t launch_read(const ReadParams& p, cudaStream_t stream) {
  const CacheGeom& c = p.v.geom;
  const long long n = (long long)p.batch * p.num_rows * c.Hkv * (c.D / 8);
  if (n == 0) return cudaSuccess;
  const dim3 grid((unsigned)((n + 255) / 256), (p.out[0] && p.out[1]) ? 2 : 1), block(256);
  switch (c.bits) {
    case 2: return launch_pdl(read_kernel<2>, grid, block, 0, stream, p);
    case 4: return launch_pdl(read_kernel<4>, grid, block, 0, stream, p);
    case 8: return launch_pdl(read_kernel<8>, grid, block, 0, stream, p);
    default: return launch_pdl(read_kernel<16>, grid, block, 0, stream, p);
  }
}

}  // namespace kvq
