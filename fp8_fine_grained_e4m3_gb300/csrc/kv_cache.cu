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
// Measured on the device: 5 prompts of up to 4097 tokens, 8 heads of 128 (60 MB), 14.1 us from
// DRAM (4.2 TB/s: offsets, lengths and table are read one after the other before the first
// row is asked for) and 10.7 us from the L2; 3.4 us for one token of each of 64 sequences.
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

constexpr int kWarps = 8;
constexpr int kPieces = 8;  // 8-element pieces of new rows a lane holds

// Tiles (of one head's keys) that a sequence with n new tokens at `start` touches.
__device__ __forceinline__ int tiles_touched(int start, int n, int log_block) {
  return n > 0 ? ((start + n - 1) >> log_block) - (start >> log_block) + 1 : 0;
}

// New tokens and their place in sequence b; n = 0 and the status where its
// offsets or its length are out of range.
struct Span {
  int t0, n, start;
};
__device__ __forceinline__ Span span(const KvAppendArgs& a, int b, int* status) {
  Span s = {0, 0, 0};
  const int len = a.lens[b];
  bool ok = sequence_tokens(a.cu, b, a.B, a.T, a.max_new, &s.t0, &s.n);
  s.start = len - s.n;
  ok = ok && s.start >= 0 && (long long)len <= (long long)a.width * a.block;
  if (!ok) {
    s.n = 0;
    raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
  }
  return s;
}

// A tile that a sequence touches, of its keys or values, is the work of `wpt`
// neighbouring warps (1, 2, 4 or 8: enough for the rows it can get), so that a
// whole tile's new rows are in registers at once.  Item i is (i / 2 / heads, i / 2 %
// heads), keys or values in turn, of the call's tiles: with `slots` places for each
// sequence where that wastes few (slots > 0), else found by a running sum
// over the sequences, which a warp takes 32 at a time (prompts of up to 4097
// tokens, 5 sequences: 22 us with places for the longest, 19 by the sum).
template <int kTpr, bool kE5M2>
__global__ void __launch_bounds__(32 * kWarps) kv_append_kernel(const KvAppendArgs a, int slots,
                                                                int log_wpt, int* status) {
  __shared__ float red[kWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int wpt = 1 << log_wpt;
  griddep_launch_dependents();
  griddep_wait();
  const long long item = ((long long)blockIdx.x * kWarps + warp) >> log_wpt;
  const bool is_v = item & 1;
  const int head = int((item >> 1) % a.heads);
  const long long place = (item >> 1) / a.heads;
  int b = -1, slot = 0;
  Span s = {0, 0, 0};
  if (slots > 0) {
    if (place < (long long)a.B * slots) {
      b = int(place / slots);
      slot = int(place - (long long)b * slots);
      s = span(a, b, status);
    }
  } else {
    long long before = 0;
    for (int base = 0; base < a.B; base += 32) {
      Span mine = {0, 0, 0};
      if (base + lane < a.B) mine = span(a, base + lane, status);
      const int tiles = tiles_touched(mine.start, mine.n, a.log_block);
      int upto = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, place < before + upto);
      if (past != 0u) {
        const int l = __ffs(past) - 1;
        b = base + l;
        slot = int(place - before) - __shfl_sync(0xffffffffu, upto - tiles, l);
        s.t0 = __shfl_sync(0xffffffffu, mine.t0, l);
        s.n = __shfl_sync(0xffffffffu, mine.n, l);
        s.start = __shfl_sync(0xffffffffu, mine.start, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  const int t0 = s.t0, start = s.start;
  int r0 = 0, r1 = 0, base = 0, blk = -1;
  if (b >= 0 && slot < tiles_touched(start, s.n, a.log_block)) {
    const int j = (start >> a.log_block) + slot;  // block of the sequence
    base = j << a.log_block;                      // its first token
    r0 = max(start - base, 0);
    r1 = min(start + s.n - base, a.block);
    blk = a.table[size_t(b) * a.width + j];
    if (blk < 0 || blk >= a.num_blocks) {
      r1 = r0 = 0;
      if (lane == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    }
  }
  const bool work = r0 < r1;  // the same for all warps of a tile
  constexpr int dim = 8 * kTpr;
  const size_t tile = work ? size_t(blk) * a.heads + head : 0;
  uint8_t* codes = (is_v ? a.vc : a.kc) + tile * a.block * dim;
  float* scale = (is_v ? a.vs : a.ks) + tile;
  const __nv_bfloat16* X = is_v ? a.V : a.K;
  const long long ld = is_v ? a.ld_v : a.ld_k;

  constexpr int kRowsAtOnce = 32 / kTpr;  // rows a warp covers with one piece a lane
  const int part = warp & (wpt - 1), col = lane % kTpr * 8;
  const int row = r0 + part * kRowsAtOnce + lane / kTpr, step = kRowsAtOnce << log_wpt;
  Raw8<__nv_bfloat16> x[kPieces];
  float old = 0.f;
  if (work) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      zero8(x[i]);
      if (row + i * step < r1) x[i] = load8(X + (t0 + base + row + i * step - start) * ld + head * dim + col);
    }
    if (r0 > 0) old = *scale;
  }
  float amax = 0.f;
  if (work) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float v[8];
      unpack8(x[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  if (wpt > 1) {
    if (lane == 0) red[warp] = amax;
    __syncthreads();  // also: every warp of the tile has read the old scale
    for (int w = 0; w < wpt; ++w) amax = fmaxf(amax, red[warp - part + w]);
  }
  if (!work) return;
  const float scale_now = fmaxf(old, pow2_scale<kE5M2>(amax));
  // A power of two (the reciprocal of one in this range is a normal number): the
  // product with the reciprocal is the quotient, exactly.  A cache filled by
  // other means may hold any scale.
  const uint32_t bits = __float_as_uint(scale_now);
  const bool pow2 = (bits & 0x807fffffu) == 0u && bits >= 1u << 23 && bits <= 253u << 23;
  const float inv = pow2 ? __uint_as_float((254u << 23) - bits) : 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (row + i * step >= r1) continue;
    float v[8];
    unpack8(x[i], v);
    uint2 q = make_uint2(0u, 0u);
    if (pow2) {
      q.x = cvt_f8x2<kE5M2>(v[0] * inv, v[1] * inv) | (cvt_f8x2<kE5M2>(v[2] * inv, v[3] * inv) << 16);
      q.y = cvt_f8x2<kE5M2>(v[4] * inv, v[5] * inv) | (cvt_f8x2<kE5M2>(v[6] * inv, v[7] * inv) << 16);
    } else if (scale_now != 0.f) {
      q.x = quant4<kE5M2>(make_float4(v[0], v[1], v[2], v[3]), scale_now);
      q.y = quant4<kE5M2>(make_float4(v[4], v[5], v[6], v[7]), scale_now);
    }
    *reinterpret_cast<uint2*>(codes + (row + i * step) * dim + col) = q;
  }
  if (scale_now > old || r0 == 0) {
    if (part == 0 && lane == 0) *scale = scale_now;
    const float ratio = scale_now != 0.f ? __fdiv_rn(old, scale_now) : 1.f;
    for (int r = row - r0; r < r0; r += step) {
      uint2* p = reinterpret_cast<uint2*>(codes + r * dim + col);
      const uint2 q = *p;
      *p = make_uint2(rescale4<kE5M2>(q.x, ratio), rescale4<kE5M2>(q.y, ratio));
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const LaunchCtx& c, const KvAppendArgs& a) {
  const int slots = (a.max_new + a.block - 2) / a.block + 1;
  int log_wpt = 0;
  while (min(a.block, a.max_new) * a.dim > 32 * 8 * kPieces << log_wpt) ++log_wpt;
  // tiles of one head: at most `slots` a sequence, and at most two a sequence that its tokens do
  // not fill
  const long long by_slots = (long long)a.B * slots, by_tokens = a.T / a.block + 2LL * a.B;
  const bool search = by_slots > 2 * by_tokens;
  const long long items = 2 * a.heads * (search ? by_tokens : by_slots);
  const long long grid = ((items << log_wpt) + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  auto fn = a.dim == 128 ? (e5 ? kv_append_kernel<16, true> : kv_append_kernel<16, false>)
                         : (e5 ? kv_append_kernel<8, true> : kv_append_kernel<8, false>);
  return launch_dependent(c, fn, unsigned(grid), 32 * kWarps, 0, a, search ? 0 : slots, log_wpt,
                          c.status);
}

}  // namespace fp8gemm
