// kv_cache.cu -- new keys and values into a paged FP8 cache.
//
// The cache holds blocks of `block` tokens; a (block, head) tile is block x dim
// FP8 bytes in a row with one FP32 scale.  For the tokens that enter a tile:
//   need = the smallest power of two >= amax / limit (at least 2^-126; 0 for zeros)
//   s    = need for a tile whose first token is new, else max(s, need)
//   code = f8(x / s);  where s grew, the tokens already there become f8(code s_old / s)
// FP8 is a floating format, so a power of two costs no precision against
// amax / limit itself, and moving a tile to a larger one only shifts exponents:
// exact but for codes that reach the subnormals.
//
// Bound by memory for prompts (2 bytes read and 1 written per element) and by
// latency for single tokens: a tile's new rows are read once, into registers.
#include "common.cuh"
#include "f8_convert.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

// amax / limit up to a power of two.
template <bool kE5M2>
__device__ __forceinline__ float pow2_scale(float amax) {
  if (amax == 0.f) return 0.f;
  const uint32_t u = __float_as_uint(__fdiv_rn(amax, f8_limit<kE5M2>()));
  const uint32_t up = (u + 0x007fffffu) & 0x7f800000u;  // the next exponent unless the mantissa is 0
  return __uint_as_float(max(up, 0x00800000u));
}

// Four codes times a power of two <= 1, rounded again.
template <bool kE5M2>
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
  const float2 lo = f8x2_to_float2<kE5M2>(uint16_t(codes));
  const float2 hi = f8x2_to_float2<kE5M2>(uint16_t(codes >> 16));
  return cvt_f8x2<kE5M2>(lo.x * ratio, lo.y * ratio) |
         (cvt_f8x2<kE5M2>(hi.x * ratio, hi.y * ratio) << 16);
}

constexpr int kMaxRowsInFlight = 8;  // 128 rows of 128 elements on 256 threads

// Grid (slots, heads, 2 B): the slot-th tile that sequence z / 2 touches, of
// its keys (z even) or values.  kTpr threads cover a row of 8 kTpr elements.
template <int kTpr, bool kE5M2>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a, int* status) {
  __shared__ float red[8];
  const int b = blockIdx.z >> 1, head = blockIdx.y, is_v = blockIdx.z & 1;
  int t0 = 0, n = 0;
  if (!sequence_tokens(a.cu, b, a.B, a.T, a.max_new, &t0, &n)) {
    if (threadIdx.x == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    return;
  }
  if (n == 0) return;
  const int len = a.lens[b], start = len - n;
  if (start < 0 || (long long)len > (long long)a.width * a.block) {
    if (threadIdx.x == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    return;
  }
  const int j = start / a.block + blockIdx.x;  // block of the sequence
  const int base = j * a.block;                // its first token
  const int r0 = max(start - base, 0), r1 = min(len - base, a.block);
  if (r0 >= r1) return;
  const int blk = a.table[size_t(b) * a.width + j];
  if (blk < 0 || blk >= a.num_blocks) {
    if (threadIdx.x == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    return;
  }
  constexpr int dim = 8 * kTpr;
  const size_t tile = size_t(blk) * a.heads + head;
  uint8_t* codes = (is_v ? a.vc : a.kc) + tile * a.block * dim;
  float* scale = (is_v ? a.vs : a.ks) + tile;
  const __nv_bfloat16* X = is_v ? a.V : a.K;
  const long long ld = is_v ? a.ld_v : a.ld_k;

  const int lane_row = threadIdx.x / kTpr, col = threadIdx.x % kTpr * 8;
  const int rows = blockDim.x / kTpr;
  Raw8<__nv_bfloat16> x[kMaxRowsInFlight];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxRowsInFlight; ++i) {
    const int r = r0 + lane_row + i * rows;
    zero8(x[i]);
    if (r < r1) x[i] = load8(X + (t0 + base + r - start) * ld + head * dim + col);
  }
  const float old = r0 > 0 ? *scale : 0.f;
#pragma unroll
  for (int i = 0; i < kMaxRowsInFlight; ++i) {
    float v[8];
    unpack8(x[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = amax;
  __syncthreads();  // also: every thread has read the old scale
  for (int w = 0; w < blockDim.x / 32; ++w) amax = fmaxf(amax, red[w]);
  const float need = pow2_scale<kE5M2>(amax);
  const float s = fmaxf(old, need);
#pragma unroll
  for (int i = 0; i < kMaxRowsInFlight; ++i) {
    const int r = r0 + lane_row + i * rows;
    if (r >= r1) continue;
    float v[8];
    unpack8(x[i], v);
    uint2 q = make_uint2(0u, 0u);
    if (s != 0.f) {
      q.x = quant4<kE5M2>(make_float4(v[0], v[1], v[2], v[3]), s);
      q.y = quant4<kE5M2>(make_float4(v[4], v[5], v[6], v[7]), s);
    }
    *reinterpret_cast<uint2*>(codes + r * dim + col) = q;
  }
  if (s > old || r0 == 0) {
    if (threadIdx.x == 0) *scale = s;
    const float ratio = s != 0.f ? __fdiv_rn(old, s) : 1.f;
    for (int r = lane_row; r < r0; r += rows) {
      uint2* p = reinterpret_cast<uint2*>(codes + r * dim + col);
      const uint2 q = *p;
      *p = make_uint2(rescale4<kE5M2>(q.x, ratio), rescale4<kE5M2>(q.y, ratio));
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const LaunchCtx& c, const KvAppendArgs& a) {
  const int tpr = a.dim / 8;
  const int rows = min(a.block, a.max_new);
  // enough threads for the rows one tile can get: 8 a thread at most
  const int threads = min(256, ceil_div(rows * tpr, 32) * 32);
  const dim3 grid((a.max_new + a.block - 2) / a.block + 1, a.heads, 2 * a.B);
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  auto fn = a.dim == 128 ? (e5 ? kv_append_kernel<16, true> : kv_append_kernel<16, false>)
                         : (e5 ? kv_append_kernel<8, true> : kv_append_kernel<8, false>);
  fn<<<grid, threads, 0, c.stream>>>(a, c.status);
  return cudaGetLastError();
}

}  // namespace fp8gemm
