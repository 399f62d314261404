// norm.cu -- root-mean-square norm with the residual's addition and an FP8
// output in 1x128 blocks, and its gradient.
//
//   h = x + r (rounded to the stream's type),  rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h rstd g,  s = max |y| / limit per 1x128 block,  q = f8(y / s)
//
//   dx = rstd (dy g - xhat mean(dy g xhat)) + dh,  dg = sum over rows of dy xhat
//   with xhat = h rstd  (the quantiser passes the gradient straight through)
//
// Both are bound by memory: a row is read once into registers, reduced there
// and written once.  Sums and statistics are FP32.
#include "common.cuh"
#include "f8_convert.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

// Sum of v over the CTA's threads, the same bits in every thread; red holds 32 floats.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = warp_sum(v);
  const int warps = (blockDim.x + 31) / 32;
  if (warps == 1) return v;
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  const int lane = threadIdx.x % 32;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// One CTA per row; thread t holds elements 8 (t + i blockDim.x) .. + 7 for i < kIter.
// A 1x128 block is 16 neighbouring threads.
template <class T, int kIter, bool kE5M2, bool kRes>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(
    const T* __restrict__ X, const T* R, const float* __restrict__ G, float eps, T* H,
    uint8_t* __restrict__ Q, float* __restrict__ sQ, float* __restrict__ rstd_out, int K) {
  __shared__ float red[32];
  const size_t row = size_t(blockIdx.x) * K;
  const int Kb = ceil_div(K, kBlockK);
  float h[kIter][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    Raw8<T> x;
    zero8(x);
    if (k < K) x = load8(X + row + k);
    unpack8(x, h[i]);
    if constexpr (kRes) {
      Raw8<T> r;
      zero8(r);
      if (k < K) r = load8(R + row + k);
      float rv[8];
      unpack8(r, rv);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] += rv[j];
      pack8(h[i], x);  // what the gradient and the next layer see
      unpack8(x, h[i]);
      if (k < K) store8(H + row + k, x);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += h[i][j] * h[i][j];
  }
  const float rstd = __frsqrt_rn(__fdiv_rn(cta_sum(sum, red), float(K)) + eps);
  if (threadIdx.x == 0 && rstd_out) rstd_out[blockIdx.x] = rstd;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    float g[8] = {};
    if (k < K) unpack8(load8(G + k), g);
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = h[i][j] * rstd * g[j];
      amax = fmaxf(amax, fabsf(h[i][j]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = __fdiv_rn(amax, f8_limit<kE5M2>());
    if (k < K) {
      uint2 q = make_uint2(0u, 0u);
      if (amax != 0.f) {
        q.x = quant4<kE5M2>(make_float4(h[i][0], h[i][1], h[i][2], h[i][3]), s);
        q.y = quant4<kE5M2>(make_float4(h[i][4], h[i][5], h[i][6], h[i][7]), s);
      }
      *reinterpret_cast<uint2*>(Q + row + k) = q;
      if (threadIdx.x % 16 == 0) sQ[size_t(blockIdx.x) * Kb + k / kBlockK] = s;
    }
  }
}

// CTA c takes rows c, c + gridDim.x, ...; thread t owns columns
// 8 (t + i blockDim.x) .. + 7 of every one of them, so its share of the gain's
// gradient stays in registers until the CTA leaves it in row c of `part`.
template <class T, int kIter, bool kRes>
__global__ void __launch_bounds__(1024) rmsnorm_backward_kernel(
    const T* __restrict__ dY, const T* __restrict__ H, const float* __restrict__ rstd_in,
    const float* __restrict__ G, const T* dH, T* dX, float* __restrict__ part, int M, int K) {
  __shared__ float red[2][32];
  float g[kIter][8], dg[kIter][8];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[i][j] = dg[i][j] = 0.f;
    if (k < K) unpack8(load8(G + k), g[i]);
  }
  int flip = 0;  // two buffers: a row's sums are read while the next row's are written
  for (int m = blockIdx.x; m < M; m += gridDim.x, flip ^= 1) {
    const size_t row = size_t(m) * K;
    const float rstd = rstd_in[m];
    float xh[kIter][8], dx[kIter][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      Raw8<T> h, dy;
      zero8(h);
      zero8(dy);
      if (k < K) {
        h = load8(H + row + k);
        dy = load8(dY + row + k);
      }
      unpack8(h, xh[i]);
      unpack8(dy, dx[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rstd;
        dg[i][j] += dx[i][j] * xh[i][j];
        dx[i][j] *= g[i][j];
        sum += dx[i][j] * xh[i][j];
      }
    }
    const float c = __fdiv_rn(cta_sum(sum, red[flip]), float(K));
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      if (k >= K) continue;
      float up[8] = {};
      if constexpr (kRes) unpack8(load8(dH + row + k), up);
#pragma unroll
      for (int j = 0; j < 8; ++j) dx[i][j] = (dx[i][j] - xh[i][j] * c) * rstd + up[j];
      Raw8<T> o;
      pack8(dx[i], o);
      store8(dX + row + k, o);
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    if (k >= K) continue;
    Raw8<float> o;
    pack8(dg[i], o);
    store8(part + size_t(blockIdx.x) * K + k, o);
  }
}

// dG[k] = sum over the rows of part [P, K], in row order within each of 32
// interleaved shares and over the shares: the same order on every run.
__global__ void __launch_bounds__(1024) gain_reduce_kernel(const float* __restrict__ part,
                                                           float* __restrict__ dG, int P, int K) {
  __shared__ float s[32][33];
  const int k = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (k < K)
    for (int p = threadIdx.y; p < P; p += 32) v += part[size_t(p) * K + k];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int kk = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && kk < K) dG[kk] = v;
}

// Threads of a row's CTA, and 8-element chunks a thread holds (K <= kMaxNormK).
void row_shape(int K, int* threads, int* iter) {
  const int chunks = ceil_div(K, 8);
  *iter = chunks > 1024 ? 2 : 1;
  *threads = ceil_div(ceil_div(chunks, *iter), 32) * 32;
}

template <class T, int kIter>
cudaError_t launch_fwd(const LaunchCtx& c, const NormArgs& a, int threads) {
  const T* X = static_cast<const T*>(a.X);
  const T* R = static_cast<const T*>(a.R);
  T* H = static_cast<T*>(a.H);
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  auto fn = R ? (e5 ? rmsnorm_quant_kernel<T, kIter, true, true>
                    : rmsnorm_quant_kernel<T, kIter, false, true>)
              : (e5 ? rmsnorm_quant_kernel<T, kIter, true, false>
                    : rmsnorm_quant_kernel<T, kIter, false, false>);
  fn<<<a.M, threads, 0, c.stream>>>(X, R, a.G, a.eps, H, a.Q, a.sQ, a.rstd, a.K);
  return cudaGetLastError();
}

template <class T, int kIter>
cudaError_t launch_bwd(const LaunchCtx& c, const NormGradArgs& a, int threads, int grid,
                       float* part) {
  auto fn = a.dH ? rmsnorm_backward_kernel<T, kIter, true> : rmsnorm_backward_kernel<T, kIter, false>;
  fn<<<grid, threads, 0, c.stream>>>(static_cast<const T*>(a.dY), static_cast<const T*>(a.H),
                                     a.rstd, a.G, static_cast<const T*>(a.dH),
                                     static_cast<T*>(a.dX), part, a.M, a.K);
  if (cudaError_t e = cudaGetLastError()) return e;
  gain_reduce_kernel<<<ceil_div(a.K, 32), dim3(32, 32), 0, c.stream>>>(part, a.dG, grid, a.K);
  return cudaGetLastError();
}

int bwd_grid(const LaunchCtx& c, int M, int threads) {
  return min(M, c.num_sms * max(1, 1536 / threads));
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const LaunchCtx& c, const NormArgs& a) {
  int threads, iter;
  row_shape(a.K, &threads, &iter);
  switch (iter) {
    case 1: return a.f32 ? launch_fwd<float, 1>(c, a, threads) : launch_fwd<__nv_bfloat16, 1>(c, a, threads);
    default: return a.f32 ? launch_fwd<float, 2>(c, a, threads) : launch_fwd<__nv_bfloat16, 2>(c, a, threads);
  }
}

size_t rmsnorm_backward_workspace_bytes(const LaunchCtx& c, int M, int K) {
  int threads, iter;
  row_shape(K, &threads, &iter);
  return size_t(bwd_grid(c, M, threads)) * K * 4;
}

cudaError_t launch_rmsnorm_backward(const LaunchCtx& c, const NormGradArgs& a, void* ws) {
  int threads, iter;
  row_shape(a.K, &threads, &iter);
  const int grid = bwd_grid(c, a.M, threads);
  float* part = static_cast<float*>(ws);
  switch (iter) {
    case 1:
      return a.f32 ? launch_bwd<float, 1>(c, a, threads, grid, part)
                   : launch_bwd<__nv_bfloat16, 1>(c, a, threads, grid, part);
    default:
      return a.f32 ? launch_bwd<float, 2>(c, a, threads, grid, part)
                   : launch_bwd<__nv_bfloat16, 2>(c, a, threads, grid, part);
  }
}

}  // namespace fp8gemm
