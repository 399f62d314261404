// moe_few.cu -- a whole mixture-of-experts layer for a few tokens (T <= 64).
//
//   ids, w  the top k logits of each token (ties to the lowest index) and their
//           softmax, over the chosen (renormalise) or over all experts
//   h       f8 1x128 of silu(x W1_gate^T) * (x W1_up^T)    per (token, choice)
//   out     sum over the choices of w * h W2^T, in BF16
//
// with x and the weights in FP8 as the GEMMs take them (1x128 and 128x128
// scales; each K block's partial product is multiplied by its scale product
// and added in FP32).
//
// Bound by the chosen experts' weights, read once: they go straight from
// memory into the registers of the m16n8k32 fragment they belong to (weight
// rows are the 16-row side, tokens the 8-column side).  A contraction's order
// is free, so k is dealt to the fragments such that a lane's share of a row's
// K block is two runs of 16 bytes.
#include "common.cuh"
#include "f8_convert.cuh"
#include "moe_few.cuh"
#include "ptx.cuh"

namespace fp8gemm {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's share of one row's K block: bytes 16 t .. + 15 and 64 + 16 t .. + 15;
// zeros past the row's K bytes (K is a multiple of 16).
struct Chunk {
  uint32_t w[8];
};
__device__ __forceinline__ Chunk load_chunk(const uint8_t* row, int k0, int K, int t) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = k0 + 64 * i + 16 * t;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row != nullptr && k < K) v = __ldg(reinterpret_cast<const uint4*>(row + k));
    c.w[4 * i] = v.x;
    c.w[4 * i + 1] = v.y;
    c.w[4 * i + 2] = v.z;
    c.w[4 * i + 3] = v.w;
  }
  return c;
}

// One K block of 16 weight rows (lo: rows 0-7, hi: rows 8-15) times 8 tokens.
__device__ __forceinline__ void mma_block(float (&d)[4], const Chunk& lo, const Chunk& hi,
                                          const Chunk& x) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    mma_e4m3(d, lo.w[2 * s], hi.w[2 * s], lo.w[2 * s + 1], hi.w[2 * s + 1], x.w[2 * s],
             x.w[2 * s + 1]);
}

// ------------------------------------------------------------------ routing
// One CTA: a warp per token chooses the experts; then a thread per expert
// lists its (token, choice) pairs in order.
__global__ void __launch_bounds__(1024) moe_route_kernel(const float* __restrict__ logits,
                                                         MoeRoute r, int32_t* ids_out,
                                                         float* w_out, int T, int E, int k,
                                                         int renormalise) {
  __shared__ int ids[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ int active;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) active = 0;
  for (int t = warp; t < T; t += blockDim.x / 32) {
    constexpr int kPer = kMoeMaxExperts / 32;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < E ? logits[t * E + e] : -INFINITY;
      if (isnan(v[i])) v[i] = -INFINITY;
    }
    uint32_t taken = 0;  // bit i: this lane's expert lane + 32 i is chosen (or not there)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i >= E) taken |= 1u << i;
    float first = 0.f, sum = 0.f, mine = 0.f;
    for (int j = 0; j < k; ++j) {
      float best = -INFINITY;
      int at = kMoeMaxExperts;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        if (!(taken >> i & 1) && (at == kMoeMaxExperts || v[i] > best)) {
          best = v[i];
          at = e;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float ob = __shfl_xor_sync(0xffffffffu, best, o);
        const int oa = __shfl_xor_sync(0xffffffffu, at, o);
        if (oa < kMoeMaxExperts &&
            (at == kMoeMaxExperts || ob > best || (ob == best && oa < at))) {
          best = ob;
          at = oa;
        }
      }
      if (at % 32 == lane) taken |= 1u << (at / 32);
      if (j == 0) first = best;
      const float p = best == -INFINITY ? 0.f : expf(best - first);
      sum += p;
      if (j == lane) mine = p;
      if (lane == 0) ids[t * k + j] = at;
      if (j == lane) ids_out[t * k + j] = at;
    }
    if (!renormalise) {  // over all experts
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += v[i] == -INFINITY ? 0.f : expf(v[i] - first);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < k) {
      const float w = sum > 0.f ? __fdiv_rn(mine, sum) : 0.f;
      w_out[t * k + lane] = w;
      r.weight[t * k + lane] = w;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int n = 0;
    for (int p = 0; p < T * k; ++p)
      if (ids[p] == e) r.pairs[e * T + n++] = p;
    r.count[e] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    for (int e = 0; e < E; ++e)
      if (r.count[e] > 0) r.expert[n++] = e;
    *r.active = n;
  }
}

// ------------------------------------------------- gate and up products, SwiGLU
// Grid (I / 16, experts at most): rows i0 .. i0 + 15 of gate and up of the
// y-th chosen expert, for all its tokens.  The warps share the K blocks.
template <int NT>
__global__ void __launch_bounds__(32 * kWarps) moe_up_kernel(const MoeArgs a, const MoeRoute r,
                                                             float* __restrict__ Hf) {
  __shared__ float part[kWarps][2][NT][4][32];
  if (int(blockIdx.y) >= *r.active) return;
  const int e = r.expert[blockIdx.y], cnt = r.count[e];
  const int i0 = blockIdx.x * 16;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int Kb = ceil_div(a.H, kBlockK);
  const uint8_t* W = a.W1 + size_t(e) * 2 * a.I * a.H;
  const uint8_t* rows[4] = {W + size_t(i0 + g) * a.H, W + size_t(i0 + g + 8) * a.H,
                            W + size_t(a.I + i0 + g) * a.H, W + size_t(a.I + i0 + g + 8) * a.H};
  const float* sW = a.s1 + size_t(e) * ceil_div(2 * a.I, 128) * Kb;
  const float* sg = sW + size_t(i0 / 128) * Kb;
  const float* su = sW + size_t((a.I + i0) / 128) * Kb;
  const uint8_t* x[NT];
  const float* sx[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int* list = r.pairs + e * a.T;
    x[n] = 8 * n + g < cnt ? a.A + size_t(list[8 * n + g] / a.k) * a.H : nullptr;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int p = 8 * n + 2 * t + c;
      sx[n][c] = p < cnt ? a.sA + size_t(list[p] / a.k) * Kb : nullptr;
    }
  }
  float acc[2][NT][4] = {};
  for (int kb = warp; kb < Kb; kb += kWarps) {
    Chunk w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = load_chunk(rows[i], kb * kBlockK, a.H, t);
    const float sgk = sg[kb], suk = su[kb];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= cnt) break;
      const Chunk xc = load_chunk(x[n], kb * kBlockK, a.H, t);
      float dg[4] = {}, du[4] = {};
      mma_block(dg, w[0], w[1], xc);
      mma_block(du, w[2], w[3], xc);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float s = sx[n][c] ? sx[n][c][kb] : 0.f;
        acc[0][n][c] = fmaf(dg[c], s * sgk, acc[0][n][c]);
        acc[0][n][2 + c] = fmaf(dg[2 + c], s * sgk, acc[0][n][2 + c]);
        acc[1][n][c] = fmaf(du[c], s * suk, acc[1][n][c]);
        acc[1][n][2 + c] = fmaf(du[2 + c], s * suk, acc[1][n][2 + c]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) part[warp][m][n][c][lane] = acc[m][n][c];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 128; i += 32 * kWarps) {
    // element c of lane l of fragment n: row l / 4 + 8 (c / 2), token 2 (l % 4) + c % 2
    const int n = i / 128, c = i / 32 % 4, l = i % 32;
    const int tok = 8 * n + 2 * (l % 4) + (c & 1);
    if (tok >= cnt) continue;
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      gate += part[w][0][n][c][l];
      up += part[w][1][n][c][l];
    }
    const int pair = r.pairs[e * a.T + tok];
    Hf[size_t(pair) * a.I + i0 + l / 4 + 8 * (c >> 1)] = __fdiv_rn(gate, 1.f + expf(-gate)) * up;
  }
}

// --------------------------------------------- down product and weighted sum
// One CTA per 16 output columns: it walks the chosen experts in order; its
// warps share each expert's K blocks and keep a sum per token in shared memory.
template <int NT>
__global__ void __launch_bounds__(32 * kWarps) moe_down_kernel(const MoeArgs a, const MoeRoute r,
                                                               const uint8_t* __restrict__ H8,
                                                               const float* __restrict__ sH,
                                                               __nv_bfloat16* __restrict__ D) {
  extern __shared__ float sums[];  // [kWarps][T][16]
  const int h0 = blockIdx.x * 16;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int Kb = ceil_div(a.I, kBlockK);
  for (int i = threadIdx.x; i < kWarps * a.T * 16; i += 32 * kWarps) sums[i] = 0.f;
  __syncthreads();
  float* mine = sums + warp * a.T * 16;
  const int active = *r.active;
  for (int y = 0; y < active; ++y) {
    const int e = r.expert[y], cnt = r.count[e];
    const int* list = r.pairs + e * a.T;
    const uint8_t* W = a.W2 + size_t(e) * a.H * a.I;
    const uint8_t* rows[2] = {W + size_t(h0 + g) * a.I, W + size_t(h0 + g + 8) * a.I};
    const float* sW = a.s2 + (size_t(e) * ceil_div(a.H, 128) + h0 / 128) * Kb;
    float acc[NT][4] = {};
    for (int kb = warp; kb < Kb; kb += kWarps) {
      const Chunk lo = load_chunk(rows[0], kb * kBlockK, a.I, t);
      const Chunk hi = load_chunk(rows[1], kb * kBlockK, a.I, t);
      const float sw = sW[kb];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= cnt) break;
        const uint8_t* x = 8 * n + g < cnt ? H8 + size_t(list[8 * n + g]) * a.I : nullptr;
        const Chunk xc = load_chunk(x, kb * kBlockK, a.I, t);
        float d[4] = {};
        mma_block(d, lo, hi, xc);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int p = 8 * n + 2 * t + c;
          const float s = p < cnt ? sH[size_t(list[p]) * Kb + kb] * sw : 0.f;
          acc[n][c] = fmaf(d[c], s, acc[n][c]);
          acc[n][2 + c] = fmaf(d[2 + c], s, acc[n][2 + c]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int p = 8 * n + 2 * t + c;
        if (p >= cnt) continue;
        const int pair = list[p];
        const float w = r.weight[pair];
        float* s = mine + pair / a.k * 16;
        s[g] = fmaf(acc[n][c], w, s[g]);
        s[g + 8] = fmaf(acc[n][2 + c], w, s[g + 8]);
      }
    __syncwarp();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += 32 * kWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w * a.T * 16 + i];
    D[size_t(i / 16) * a.H + h0 + i % 16] = __float2bfloat16_rn(v);
  }
}

struct Layout {
  size_t hf, h8, sh, weight, pairs, count, expert, active, total;
};

Layout layout(const MoeArgs& a) {
  const size_t P = size_t(a.T) * a.k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 15) / 16 * 16;
    return here;
  };
  Layout l;
  l.hf = take(P * a.I * 4);
  l.h8 = take(P * a.I);
  l.sh = take(P * ceil_div(a.I, kBlockK) * 4);
  l.weight = take(P * 4);
  l.pairs = take(size_t(a.E) * a.T * 4);
  l.count = take(size_t(a.E) * 4);
  l.expert = take(size_t(a.E) * 4);
  l.active = take(4);
  l.total = at;
  return l;
}

template <int NT>
cudaError_t launch_nt(const LaunchCtx& c, const MoeArgs& a, const MoeRoute& r, char* ws,
                      const Layout& l) {
  float* Hf = reinterpret_cast<float*>(ws + l.hf);
  uint8_t* H8 = reinterpret_cast<uint8_t*>(ws + l.h8);
  float* sH = reinterpret_cast<float*>(ws + l.sh);
  const int most = min(a.E, a.T * a.k);
  moe_up_kernel<NT><<<dim3(a.I / 16, most), 32 * kWarps, 0, c.stream>>>(a, r, Hf);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (cudaError_t e = launch_quant_1x128(c, Hf, H8, sH, a.T * a.k, a.I)) return e;
  moe_down_kernel<NT><<<a.H / 16, 32 * kWarps, size_t(kWarps) * a.T * 64, c.stream>>>(a, r, H8, sH, a.D);
  return cudaGetLastError();
}

}  // namespace

size_t moe_few_workspace_bytes(const MoeArgs& a) { return layout(a).total; }

cudaError_t launch_moe_few(const LaunchCtx& c, const MoeArgs& a, void* workspace, int* launches) {
  char* ws = static_cast<char*>(workspace);
  const Layout l = layout(a);
  const MoeRoute r{reinterpret_cast<float*>(ws + l.weight), reinterpret_cast<int*>(ws + l.pairs),
                   reinterpret_cast<int*>(ws + l.count), reinterpret_cast<int*>(ws + l.expert),
                   reinterpret_cast<int*>(ws + l.active)};
  moe_route_kernel<<<1, 1024, 0, c.stream>>>(a.logits, r, a.ids, a.weights, a.T, a.E, a.k,
                                             a.renormalise);
  if (cudaError_t e = cudaGetLastError()) return e;
  *launches = 4;
  if (a.T <= 8) return launch_nt<1>(c, a, r, ws, l);
  if (a.T <= 16) return launch_nt<2>(c, a, r, ws, l);
  if (a.T <= 32) return launch_nt<4>(c, a, r, ws, l);
  return launch_nt<8>(c, a, r, ws, l);
}

}  // namespace fp8gemm
