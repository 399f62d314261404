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
// and written once.  Sums and statistics are FP32.  Measured, BF16 with a residual:
// 4096 x 7168 forward 36.6 us, 5.6 TB/s; 8192 x 4096 backward 46.3 us, 5.8 TB/s.
#include <cfloat>

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

// The larger value, or NaN if one is: a NaN in a block must not look like the others' maximum
// (a diverged row would become codes and scales of 0).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// amax / limit: the corrected quotient where that is exact.
template <bool kE5M2>
__device__ __forceinline__ float block_scale(float amax) {
  constexpr float kLimit = kE5M2 ? 57344.f : 448.f;
  const Reciprocal d{kLimit, 1.f / kLimit, true};
  return amax >= 1e-25f && amax <= 1e30f ? quotient(amax, d) : __fdiv_rn(amax, kLimit);
}

// Eight values to codes of one scale; zeros where it is 0 (all zeros, or a maximum so
// small that the scale underflows: the quotient of a 0 there would be NaN).
template <bool kE5M2>
__device__ __forceinline__ uint2 quant8(const float (&v)[8], const Reciprocal& d) {
  const float4 a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
  if (d.safe) return make_uint2(quant4<kE5M2>(a, d), quant4<kE5M2>(b, d));
  if (d.s == 0.f) return make_uint2(0u, 0u);
  return make_uint2(quant4<kE5M2>(a, d.s), quant4<kE5M2>(b, d.s));
}

// One CTA per row; thread t holds elements 8 (t + i blockDim.x) .. + 7 for i < kIter.
// A 1x128 block is 16 neighbouring threads.
// CTAs that stay and take row after row, the next one asked for ahead, were slower
// (4096 x 7168: 39 us and more): the CTAs' starts already overlap.
template <class T, int kIter, bool kE5M2, bool kRes>
__global__ void __launch_bounds__(kIter == 4 ? 512 : 1024) rmsnorm_quant_kernel(
    const T* __restrict__ X, const T* R, const float* __restrict__ G, float eps, T* H,
    uint8_t* __restrict__ Q, float* __restrict__ sQ, float* __restrict__ rstd_out, int K) {
  __shared__ float red[2][32];
  const size_t row = size_t(blockIdx.x) * K;
  const int Kb = ceil_div(K, kBlockK);
  griddep_launch_dependents();
  griddep_wait();
  Raw8<T> x[kIter], r[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    zero8(x[i]);
    zero8(r[i]);
    if (k < K) {
      x[i] = load8(X + row + k);
      if constexpr (kRes) r[i] = load8(R + row + k);
    }
  }
  float h[kIter][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if constexpr (kRes) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      x[i] = add8(x[i], r[i]);  // what the gradient and the next layer see
      if (k < K) store8(H + row + k, x[i]);
    }
    unpack8(x[i], h[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(h[i][j], h[i][j], sum);
  }
  sum = cta_sum(sum, red[0]);
  const float square = __fdiv_rn(sum, float(K)) + eps;
  float rstd = __frsqrt_rn(square), ry = rstd;
  // The squares leave FP32's range (|h| above 1e17; or, with next to no eps, below 1e-15): from
  // here on h times a power of two.  A row of zeros gives zeros whatever eps.
  if (!(sum <= FLT_MAX) || square < 0x1p-100f) {  // the same in every thread
    const float f = sum > 1.f ? 0x1p-100f : 0x1p100f;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] *= f;
        sum = fmaf(h[i][j], h[i][j], sum);
      }
    sum = cta_sum(sum, red[1]);
    ry = __frsqrt_rn(__fdiv_rn(sum, float(K)) + eps * f * f);
    rstd = ry * f;
    if (sum == 0.f) ry = 0.f;
  }
  if (threadIdx.x == 0 && rstd_out) rstd_out[blockIdx.x] = rstd;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    float g[8] = {};
    if (k < K) unpack8(load8(G + k), g);
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[i][j] = h[i][j] * ry * g[j];
      amax = max_nan(amax, fabsf(h[i][j]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const Reciprocal s = reciprocal(block_scale<kE5M2>(amax));
    if (k < K) {
      *reinterpret_cast<uint2*>(Q + row + k) = quant8<kE5M2>(h[i], s);
      if (threadIdx.x % 16 == 0) sQ[size_t(blockIdx.x) * Kb + k / kBlockK] = s.s;
    }
  }
}

// CTA c takes rows c, c + gridDim.x, ...; thread t owns columns
// 8 (t + i blockDim.x) .. + 7 of every one of them, so its share of the gain's
// gradient stays in registers until the CTA leaves it in row c of `part`.  The
// next row is asked for before this one is used.  CTAs that stay keep the partial
// gains few (one row of them for each CTA, 2 to 5 MB); one CTA a row would write as
// many bytes of them as it reads of the row.
template <class T, int kIter, bool kRes>
__global__ void __launch_bounds__(512) rmsnorm_backward_kernel(
    const T* dY, const T* __restrict__ H, const float* __restrict__ rstd_in,
    const float* __restrict__ G, const T* dH, T* dX, float* __restrict__ part, int M, int K) {
  __shared__ float red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  struct Row {
    Raw8<T> dy[kIter], h[kIter], up[kIter];
    float rstd;
  } next;
  auto load = [&](int m) {
    const size_t row = size_t(m) * K;
    next.rstd = rstd_in[m];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      zero8(next.dy[i]);
      zero8(next.h[i]);
      zero8(next.up[i]);
      if (k < K) {
        next.dy[i] = load8(dY + row + k);
        next.h[i] = load8(H + row + k);
        if constexpr (kRes) next.up[i] = load8(dH + row + k);
      }
    }
  };
  constexpr bool kAhead = kIter < 4;  // else a thread's registers hold one row only
  if (int(blockIdx.x) < M) load(blockIdx.x);
  float dg[kIter][8];
  Raw8<float> g[kAhead ? kIter : 1];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = 0.f;
    if constexpr (kAhead) {
      zero8(g[i]);
      if (k < K) g[i] = load8(G + k);
    }
  }
  auto gain = [&](int i, float (&v)[8]) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    if constexpr (kAhead) {
      unpack8(g[i], v);
    } else {
      Raw8<float> r;
      zero8(r);
      if (k < K) r = load8(G + k);
      unpack8(r, v);
    }
  };
  int flip = 0;  // two buffers: a row's sums are read while the next row's are written
  for (int m = blockIdx.x; m < M; m += gridDim.x, flip ^= 1) {
    float xh[kIter][8], dx[kIter][8];  // h rstd and dy g, kept over the row's sum
    Raw8<T> up[kIter];
    const float rstd = next.rstd;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      float w[8];
      unpack8(next.h[i], xh[i]);
      unpack8(next.dy[i], dx[i]);
      up[i] = next.up[i];
      gain(i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rstd;
        dg[i][j] = fmaf(dx[i][j], xh[i][j], dg[i][j]);
        dx[i][j] *= w[j];
        sum = fmaf(dx[i][j], xh[i][j], sum);
      }
    }
    if (kAhead && m + int(gridDim.x) < M) load(m + gridDim.x);
    const float c = __fdiv_rn(cta_sum(sum, red[flip]), float(K));
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      if (k >= K) continue;
      float u[8];
      unpack8(up[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dx[i][j] = fmaf(fmaf(-xh[i][j], c, dx[i][j]), rstd, kRes ? u[j] : 0.f);
      Raw8<T> o;
      pack8(dx[i], o);
      store8(dX + size_t(m) * K + k, o);
    }
    if (!kAhead && m + int(gridDim.x) < M) load(m + gridDim.x);
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
  griddep_launch_dependents();
  griddep_wait();
  if (k < K) {
#pragma unroll 8
    for (int p = threadIdx.y; p < P; p += 32) v += part[size_t(p) * K + k];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int kk = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && kk < K) dG[kk] = v;
}

// A row's CTA: iter chunks of 8 elements a thread (K <= kMaxNormK).
struct RowShape {
  int threads, iter;
};
RowShape row_shape(int chunks, int iter) { return {ceil_div(ceil_div(chunks, iter), 32) * 32, iter}; }

// A few rows want the most threads for the least latency; with rows enough for
// every SM, several chunks a thread keep more rows in flight between their barriers
// (K 7168, BF16 with a residual: 1 row 2.1 us with one chunk a thread, 3.4 with four;
// 303 rows 3.3 and 4.3; 400 rows 5.4 and 5.1; 4096 rows 41.9 and 36.6).
RowShape forward_shape(const LaunchCtx& c, int M, int K) {
  const int chunks = ceil_div(K, 8);
  if (M < 2 * c.num_sms) return row_shape(chunks, chunks > 1024 ? 2 : 1);
  return row_shape(chunks, chunks >= 256 ? 4 : chunks >= 64 ? 2 : 1);
}
RowShape backward_shape(int K) {
  const int chunks = ceil_div(K, 8);
  return row_shape(chunks, chunks > 1024 ? 4 : chunks > 256 ? 2 : 1);
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
  return launch_dependent(c, fn, a.M, threads, 0, X, R, a.G, a.eps, H, a.Q, a.sQ, a.rstd, a.K);
}

template <class T, int kIter>
cudaError_t launch_bwd(const LaunchCtx& c, const NormGradArgs& a, int threads, int grid,
                       float* part) {
  auto fn = a.dH ? rmsnorm_backward_kernel<T, kIter, true> : rmsnorm_backward_kernel<T, kIter, false>;
  if (cudaError_t e = launch_dependent(c, fn, grid, threads, 0, static_cast<const T*>(a.dY),
                                       static_cast<const T*>(a.H), a.rstd, a.G,
                                       static_cast<const T*>(a.dH), static_cast<T*>(a.dX), part,
                                       a.M, a.K))
    return e;
  return launch_dependent(c, gain_reduce_kernel, ceil_div(a.K, 32), dim3(32, 32), 0, part, a.dG, grid,
                          a.K);
}

// CTAs that run at once: 64 registers a thread with one chunk, 128 with more.
int backward_grid(const LaunchCtx& c, int M, const RowShape& s) {
  return min(M, c.num_sms * max(1, (s.iter == 1 ? 1024 : 512) / s.threads));
}

template <class T>
cudaError_t launch_fwd(const LaunchCtx& c, const NormArgs& a) {
  const RowShape s = forward_shape(c, a.M, a.K);
  switch (s.iter) {
    case 1: return launch_fwd<T, 1>(c, a, s.threads);
    case 2: return launch_fwd<T, 2>(c, a, s.threads);
    default: return launch_fwd<T, 4>(c, a, s.threads);
  }
}

template <class T>
cudaError_t launch_bwd(const LaunchCtx& c, const NormGradArgs& a, float* part) {
  const RowShape s = backward_shape(a.K);
  const int grid = backward_grid(c, a.M, s);
  switch (s.iter) {
    case 1: return launch_bwd<T, 1>(c, a, s.threads, grid, part);
    case 2: return launch_bwd<T, 2>(c, a, s.threads, grid, part);
    default: return launch_bwd<T, 4>(c, a, s.threads, grid, part);
  }
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const LaunchCtx& c, const NormArgs& a) {
  return a.f32 ? launch_fwd<float>(c, a) : launch_fwd<__nv_bfloat16>(c, a);
}

// A row of K floats for each CTA, at most kMaxNormK floats an SM (a CTA of t
// threads with i chunks has K <= 8 i t, and an SM has 1024 / t or 512 / t of them):
// the same for every call, so that a stream's buffer stays where it is.
size_t rmsnorm_backward_workspace_bytes(const LaunchCtx& c) { return size_t(c.num_sms) * kMaxNormK * 4; }

cudaError_t launch_rmsnorm_backward(const LaunchCtx& c, const NormGradArgs& a, void* ws) {
  float* part = static_cast<float*>(ws);
  return a.f32 ? launch_bwd<float>(c, a, part) : launch_bwd<__nv_bfloat16>(c, a, part);
}

}  // namespace fp8gemm
