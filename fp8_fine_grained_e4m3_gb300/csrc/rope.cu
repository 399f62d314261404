// rope.cu -- rotary positions of queries and keys, and their gradient.
//
// With t = position * freq[i] for the i-th pair (x1, x2) of a head,
//   y1 = a (x1 cos t - x2 sin t),  y2 = a (x2 cos t + x1 sin t)
// and the gradient is the same with -t (a times a rotation, transposed).  Pairs are
// elements i and i + rot / 2 of the head, or 2 i and 2 i + 1; elements past rot pass through.
//
// A far position times a frequency has more bits than FP32 holds (131072 radians would be
// known to 2^-7), so the angle is formed in FP64, in half turns, and brought into
// [-1, 1] there; its sine and cosine are FP32's (sincospi, 1 to 2 ulp).  That is ten FP64
// operations for a pair of a token, shared by all heads of the token through shared memory.
//
// Bound by memory: every element is read and written once, 16 bytes a lane.  9700 tokens of 64 + 8
// BF16 heads of 128 take 61 us, 87 % of what a plain copy reaches; the gradient of 7800 tokens of
// 32 + 8 such heads, 64 elements of each in neighbouring pairs, 29 us (80 %).  CTAs of 128
// threads and two tokens, the first loads under way before the position is looked up: CTAs of 256
// threads and eight tokens took 64 and 32 us, two units in flight a thread 64 and 31 (more registers,
// fewer threads).  A step of 64 tokens is one chain of latencies, 3.5 us.
#include "common.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxTokens = 2;  // of a CTA: a warp looks up each one's position
constexpr int kMaxPairs = kMaxRopeDim / 2;

// A token's position; false where it has none, or its sequence's offsets or length are bad (its rows are then left
// as they are).
__device__ __forceinline__ bool token_position(const RopeArgs& a, int t, int lane, int* pos) {
  if (a.positions) {
    *pos = a.positions[t];
    return true;
  }
  int b, t0, n;
  if (a.cu) {
    b = find_sequence(a.cu, a.B, t, lane);
    if (b < 0 || !sequence_tokens(a.cu, b, a.B, a.T, a.T, &t0, &n)) return false;
  } else {
    n = a.T / a.B;
    b = t / n;
    t0 = b * n;
  }
  const int len = a.lens[b];
  if (len < n) return false;
  *pos = len - n + t - t0;
  return true;
}

// Offsets and length of every sequence, whether a token finds it or not: by the warps without a token of the first CTAs.
constexpr int kFree = kThreads - 32 * kMaxTokens;
__device__ __forceinline__ void check_sequences(const RopeArgs& a, unsigned cta, int* status) {
  bool bad = false;
#pragma unroll 1
  for (long long b = (long long)cta * kFree + threadIdx.x - 32 * kMaxTokens; b < a.B;
       b += (long long)gridDim.x * gridDim.y * kFree) {
    int t0, n;
    const int len = a.lens[b];
    bad |= !sequence_tokens(a.cu, int(b), a.B, a.T, a.T, &t0, &n) | (len < n);
  }
  if (bad) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
}

template <class T>
struct Unit {  // 16 elements of a head: the two halves of 8 pairs, or 8 pairs (or none) in a row
  const T* x;
  T* y;
  int gap;    // from the first eight elements to the second eight
  int pair;   // first two pairs in the CTA's table, -1: to be copied, -2: nothing to do
  int token;  // of the CTA
};

template <class T, bool kInterleaved>
__device__ __forceinline__ void turn(const Raw8<T>& r0, const Raw8<T>& r1, const float4* cs, int gap, Raw8<T>& o0,
                                     Raw8<T>& o1) {
  float2 t[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = cs[i * gap];
    t[2 * i] = make_float2(v.x, v.y);
    t[2 * i + 1] = make_float2(v.z, v.w);
  }
  float a[8], b[8];
  unpack8(r0, a);
  unpack8(r1, b);
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = t[i], q = t[i + 4];
      const float u = a[2 * i], v = b[2 * i];
      a[2 * i] = fmaf(u, p.x, -(a[2 * i + 1] * p.y));
      a[2 * i + 1] = fmaf(a[2 * i + 1], p.x, u * p.y);
      b[2 * i] = fmaf(v, q.x, -(b[2 * i + 1] * q.y));
      b[2 * i + 1] = fmaf(b[2 * i + 1], q.x, v * q.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = t[i];
      const float u = a[i];
      a[i] = fmaf(u, p.x, -(b[i] * p.y));
      b[i] = fmaf(b[i], p.x, u * p.y);
    }
  }
  pack8(a, o0);
  pack8(b, o1);
}

// (48 registers and ten CTAs an SM in BF16, 64 and eight in FP32: with 56 registers and nine CTAs the 9700 tokens take 61.2 us
// instead of 60.3, a step 3.7 instead of 3.5.)
// CTA (x, y): tokens x tokens .. + tokens - 1, the y-th of gridDim.y shares of their heads' units.
template <class T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 10 : 8) rope_kernel(const RopeArgs a, int tokens, int* status) {
  // cos and sin, two pairs an entry: entries j of all of a token's units of 8 pairs lie in a row, so that
  // neighbouring lanes' units meet all banks
  __shared__ float4 cs[(kThreads > kMaxPairs ? kThreads : kMaxPairs) / 2];
  __shared__ int pos[kMaxTokens];
  __shared__ bool has[kMaxTokens];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t_first = blockIdx.x * tokens, n_tok = min(tokens, a.T - t_first);
  const int pairs = a.rot / 2;
  griddep_launch_dependents();
  griddep_wait();
  const int U = a.dim / 16, per_token = (a.heads_q + a.heads_k) * U;
  const int end = n_tok * per_token, step = gridDim.y * kThreads;
  auto unit = [&](int u) {
    Unit<T> r = {nullptr, nullptr, 0, -2, 0};
    if (u >= end) return r;
    const int k = u / per_token;
    u -= k * per_token;
    int h = u / U;
    const int c = u - h * U;
    const bool key = h >= a.heads_q;
    if (key) h -= a.heads_q;
    const long long t = t_first + k;
    const T* x = static_cast<const T*>(key ? a.K : a.Q) + t * (key ? a.ld_k : a.ld_q) + h * a.dim;
    T* y = static_cast<T*>(key ? a.Ko : a.Qo) + t * (key ? a.ld_ko : a.ld_qo) + h * a.dim;
    const bool turned = 16 * c < a.rot;
    if (!turned && x == y) return r;
    const bool half = turned && !kInterleaved;
    r.x = x + (half ? 8 : 16) * c;
    r.y = y + (half ? 8 : 16) * c;
    r.gap = half ? pairs : 8;
    r.pair = turned ? k * (pairs / 2) + c : -1;
    r.token = k;
    return r;
  };
  // The next unit's elements are asked for before this one's are stored; the first unit's do not
  // wait for the positions and the angles.
  Unit<T> next;
  Raw8<T> r0, r1;
  auto ask = [&](int u) {
    next = unit(u);
    zero8(r0);
    zero8(r1);
    if (next.pair != -2) {
      r0 = load8(next.x);
      r1 = load8(next.x + next.gap);
    }
  };
  int u = blockIdx.y * kThreads + threadIdx.x;
  ask(u);
  if (warp < n_tok) {
    int p = 0;
    const bool ok = token_position(a, t_first + warp, lane, &p);
    if (lane == 0) {
      pos[warp] = p;
      has[warp] = ok;
    }
  } else if (const unsigned cta = blockIdx.y * gridDim.x + blockIdx.x;
             warp >= kMaxTokens && cta <= unsigned(a.B) / kFree && !a.positions) {  // meanwhile
    check_sequences(a, cta, status);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_tok * pairs; i += kThreads) {
    const int k = i / pairs, p = i - k * pairs;
    // 1 / pi in two parts: a position of 2^31 would lose 2^-21 of a turn in one
    constexpr double kInvPi = 0.31830988618379067154, kInvPiLow = -1.9678676675182486e-17;
    const double x = double(pos[k]) * double(a.freq[p]);         // radians
    const double t = x * kInvPi;                                      // half turns
    const double low = fma(x, kInvPi, -t) + x * kInvPiLow;
    float s, c;
    sincospif(float(fma(-2.0, rint(0.5 * t), t) + low), &s, &c);
    reinterpret_cast<float2*>(cs)[k * pairs + (p % 8 / 2 * (pairs / 8) + p / 8) * 2 + p % 2] =
        make_float2(a.amplitude * c, a.backward ? -a.amplitude * s : a.amplitude * s);
  }
  __syncthreads();
  for (; u < end; u += step) {
    const Unit<T> v = next;
    Raw8<T> x0 = r0, x1 = r1;
    ask(u + step);
    if (v.pair == -2 || !has[v.token]) continue;
    if (v.pair >= 0) turn<T, kInterleaved>(x0, x1, cs + v.pair, pairs / 8, x0, x1);
    store8(v.y, x0);
    store8(v.y + v.gap, x1);
  }
}

}  // namespace

cudaError_t launch_rope(const LaunchCtx& c, const RopeArgs& a) {
  // Two tokens a CTA where that leaves two CTAs or more an SM; with few tokens one each, its heads
  // shared by as many CTAs as give an SM two (one: 3.9 us for a step of 64 tokens, two: 3.7).
  int tokens = min(kMaxTokens, max(1, kThreads / (a.rot / 2)));
  while (tokens > 1 && ceil_div(a.T, tokens) < 2 * c.num_sms) tokens /= 2;
  const int grid_x = ceil_div(a.T, tokens);
  const long long units = (long long)tokens * (a.heads_q + a.heads_k) * (a.dim / 16);
  const long long most = (units + kThreads - 1) / kThreads;
  const int grid_y = int(max(1LL, min(most, 2LL * c.num_sms / grid_x)));
  auto fn = a.f32 ? (a.interleaved ? rope_kernel<float, true> : rope_kernel<float, false>)
                  : (a.interleaved ? rope_kernel<__nv_bfloat16, true> : rope_kernel<__nv_bfloat16, false>);
  return launch_dependent(c, fn, dim3(grid_x, grid_y), kThreads, 0, a, tokens, c.status);
}

}  // namespace fp8gemm
