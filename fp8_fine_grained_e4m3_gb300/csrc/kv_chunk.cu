// kv_chunk.cu -- attention of a chunk of new tokens over the paged FP8 cache.
//
//   o = sum_j p_j v_j,  p = softmax over the visible j of (scale q . k_j)
//
// A warp for each query row: lanes are tokens for the scores, dimensions for the output.
#include <cfloat>

#include "common.cuh"
#include "f8_convert.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kWarps = 8;

template <int kDim, bool kE5M2>
__global__ void __launch_bounds__(32 * kWarps) kv_chunk_kernel(const KvChunkArgs a, int* status) {
  __shared__ float q_smem[kWarps][kDim];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int hq = a.heads * a.group;
  griddep_launch_dependents();
  griddep_wait();
  const long long row = (long long)blockIdx.x * kWarps + warp;
  if (row >= (long long)a.T * hq) return;
  const int t = int(row / hq), head = int(row % hq), hk = head / a.group;
  int b, t0, n;
  if (a.cu) {
    b = find_sequence(a.cu, a.B, t, lane);
    if (b == -1) return;
    if (b == -2 || !sequence_tokens(a.cu, b, a.B, a.T, a.max_q, &t0, &n)) {
      raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
      return;
    }
  } else {
    sequence_tokens(a.cu, t / (a.T / a.B), a.B, a.T, a.max_q, &t0, &n);
    b = t / n;
  }
  int len = a.lens[b];
  if (len < 0 || (long long)len > (long long)a.width * a.block) {
    raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    len = 0;
  }
  const int sees = a.causal ? len - n + 1 + (t - t0) : len;
  for (int d = lane; d < kDim; d += 32) q_smem[warp][d] = __bfloat162float(a.Q[t * a.ld_q + head * kDim + d]);
  __syncwarp();
  constexpr int kPer = kDim / 32;
  float o[kPer] = {}, m = -INFINITY, l = 0.f;
  for (int base = 0; base < sees; base += 32) {
    const int j = base + lane;
    float x = -INFINITY;
    int blk = -1;
    if (j < sees) {
      blk = a.table[(long long)b * a.width + j / a.block];
      if (blk < 0 || blk >= a.num_blocks) {
        raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
        blk = -1;
      }
    }
    const long long tile = (long long)blk * a.heads + hk;
    if (blk >= 0) {
      const uint8_t* k = a.kc + (tile * a.block + j % a.block) * kDim;
      float dot = 0.f;
      for (int d = 0; d < kDim; d += 2) {
        const float2 v = f8x2_to_float2<kE5M2>(*reinterpret_cast<const uint16_t*>(k + d));
        dot = fmaf(v.x, q_smem[warp][d], dot);
        dot = fmaf(v.y, q_smem[warp][d + 1], dot);
      }
      x = dot * (a.scale * a.ks[tile]);
    }
    float top = x;
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    top = fmaxf(top, m);
    if (top == -INFINITY) continue;
    const float shrink = expf(m - top), p = expf(x - top);
    m = top;
    l = l * shrink + warp_sum(p);
    for (int i = 0; i < kPer; ++i) o[i] *= shrink;
    for (int s = 0; s < 32; ++s) {
      const int blk_s = __shfl_sync(0xffffffffu, blk, s);
      const float ps = __shfl_sync(0xffffffffu, p, s);
      if (blk_s < 0) continue;
      const long long ts = (long long)blk_s * a.heads + hk;
      const uint8_t* v = a.vc + (ts * a.block + (base + s) % a.block) * kDim;
      const float f = a.vs[ts];
      for (int i = 0; i < kPer; ++i)
        o[i] = fmaf(ps, f8x2_to_float2<kE5M2>(v[lane + 32 * i]).x * f, o[i]);
    }
  }
  for (int i = 0; i < kPer; ++i)
    a.O[(row)*kDim + lane + 32 * i] = __float2bfloat16(l > 0.f || isnan(l) ? o[i] / l : 0.f);
}

}  // namespace

cudaError_t launch_kv_chunk(const LaunchCtx& c, const KvChunkArgs& a) {
  const long long rows = (long long)a.T * a.heads * a.group;
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  auto fn = a.dim == 128 ? (e5 ? kv_chunk_kernel<128, true> : kv_chunk_kernel<128, false>)
                         : (e5 ? kv_chunk_kernel<64, true> : kv_chunk_kernel<64, false>);
  return launch_dependent(c, fn, unsigned((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, a, c.status);
}

}  // namespace fp8gemm
