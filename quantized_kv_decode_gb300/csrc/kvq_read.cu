// Cached rows back to fp16 (kvq_cache_read), eight channels a thread: codes
// and headers in, fp16 rows out.  4 x 8192 tokens of 8 heads of 128, INT8
// groups of 64: 70 us, 2.9 TB/s (85 with one row a thread in flight; fp32
// conversion of eight codes a thread bounds it).
#include "kvq_load.cuh"

namespace kvq {
namespace {

// Grid: x = groups of rows (token, KV head) of a sequence, y = K / V,
// z = sequences.  A thread keeps its chunk of channels over kRows rows, whose
// loads are in flight together.
constexpr int kRows = 4;

template <int BITS>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const CacheGeom& c = p.v.geom;
  const int which = p.out[0] ? blockIdx.y : 1;
  const int chunks = c.D / 8, rpb = 256 / chunks;  // rows per pass
  const int ch = threadIdx.x % chunks, sub = threadIdx.x / chunks;
  const int all = p.num_rows * c.Hkv;
  const int first = blockIdx.x * rpb * kRows + sub;
  for (int b = blockIdx.z; b < p.batch; b += gridDim.z) {
    const int L = checked_len(c, p.seq_lens, b, -1);
    const int s0 = __ldg(p.start + b);
    uint32_t flags = 0;
    if (L < 0 || L > cache_capacity(c) || s0 < 0) {
      flags = KVQ_FLAG_SEQ_LEN;
    } else {
      uint4 x[kRows];
      bool live[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int r = first + u * rpb, t = r / c.Hkv, kvh = r - t * c.Hkv;
        live[u] = r < all && (long long)s0 + t < L;
        if (!live[u]) continue;
        const long long row = view_row(c, b, kvh, L, s0 + t);
        live[u] = row >= 0;
        if (row < 0) flags = KVQ_FLAG_BLOCK_TABLE;
        else x[u] = load8<BITS>(p.v, which, b, kvh, L, s0 + t, row, ch);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        uint4* o = reinterpret_cast<uint4*>(p.out[which]) + ((long long)b * all + first + u * rpb) * chunks + ch;
        if (live[u] && KVQ_IN(c, which ? KVQ_ARRAY_V_NEW : KVQ_ARRAY_K_NEW, o, 16)) *o = x[u];
      }
    }
    if (flags && ch == 0 && p.status) atomicOr(p.status, flags);
  }
}

}  // namespace

cudaError_t launch_read(const ReadParams& p, cudaStream_t stream) {
  const CacheGeom& c = p.v.geom;
  const long long rows = (long long)p.num_rows * c.Hkv;
  if (rows == 0 || p.batch == 0) return cudaSuccess;
  const int per = 256 / (c.D / 8) * kRows;
  const dim3 grid((unsigned)((rows + per - 1) / per), (p.out[0] && p.out[1]) ? 2 : 1,
                  (unsigned)(p.batch < 65535 ? p.batch : 65535)), block(256);
  switch (c.bits) {
    case 2: return launch_pdl(read_kernel<2>, grid, block, 0, stream, p);
    case 4: return launch_pdl(read_kernel<4>, grid, block, 0, stream, p);
    case 8: return launch_pdl(read_kernel<8>, grid, block, 0, stream, p);
    default: return launch_pdl(read_kernel<16>, grid, block, 0, stream, p);
  }
}

}  // namespace kvq
