// kv_chunk.cu -- attention of a chunk of new tokens over the paged FP8 cache (kv_cache.cu has the
// layout): prompts, chunks of them behind what is cached, queries over another sequence's states.
//
//   o = sum_j p_j v_j,  p = softmax over the visible j of (scale q . k_j)
//
// The rows of a cached head are the (token, query head of its group) pairs, in that order: they
// share every byte of it, and neighbouring rows lie side by side in Q and O.  A unit of work is
// 256 rows of one head of one sequence, in two tiles of 128, against the tokens that its last
// row sees, 128 at a time:
//   S [128, 128] = Q K^T, P = 2^(S - reference), O [128, dim] += P V
// both products by tcgen05 on FP16 operands (FP8 codes are exact in FP16; q is shifted by a power
// of two per row into its range, as BF16 has fewer bits: exact down to 2^-27 of the row's largest
// element; P has 11).  S and O live in TMEM -- the two tiles' S and O fill its 512 columns -- and P
// takes the place of S there.
//
//   warps 0-3, 4-7   softmax of tile 0 and of tile 1: thread = row = TMEM lane
//   warps 8-11       keys and values: codes to FP16, into a two-stage ring in shared memory
//                    (128-byte swizzle)
//   warp 12          issues the products: while tile 0's softmax runs, tile 1's
//                    products do
//   warp 13          finds the CTA's units and hands them on through a ring
//   warp 14          looks up where the units' tiles lie and their scales, ahead of the others
//   warp 15          asks for their codes
//
// Scales act in FP32 where they can: a key block's on the scores.  A value block's cannot act
// behind the product, whose sum runs over blocks, nor inside P or V as it is, which FP16's range
// would not take; so P carries it as a power: P = 2^(s + log2|v_scale| - reference) with the
// reference the running maximum of that sum, which is what the terms p v_scale are relative to
// the largest.  The sum of p itself is formed per block from P / |v_scale|.
//
// The reference lags behind the maximum: a first tile sets it so that its largest P is 2^kLift, and it rises (O
// is multiplied in TMEM) when 16 neighbouring P of a tile that all rows see pass 2^15 together, or one P of another
// tile.  16 such P are 2^kLift together at the least: of that sum, the row's largest, P keeps its 11 bits
// down to 2^-(14 + kLift) and is lost below 2^-(25 + kLift) (131072 tokens there are 2^-13 of the sum; the
// output is BF16).  Where a tile that some row does not see whole makes the reference rise half-way, P of its first
// tokens is multiplied by a power of two in FP32: exact, but for what FP16 then holds with fewer bits.
//
// Bound by the softmax and the chain S -> P -> O of a tile: 512 tokens x 32 heads of 128 behind 131077 take
// 0.88 ms, 1.25 PFLOP/s or 65 % of what cuBLAS reaches; a pair of tiles of rows takes 3400 cycles a tile of
// tokens, of which the tensor cores work 2200 and each softmax warp 1900 (512 of them exponentials, beside those of the
// other warp of its scheduler).  Prompts from empty caches (9 sequences, 14600 tokens x 64 heads) take 0.75 ms, 0.73
// PFLOP/s: their units are nine tiles long, and a unit's start and end cost as much as three; scores that keep rising
// cost a second pass over a tile's scores in one of four.  What the warps run together has to fit in the
// instruction cache: loops are rolled and hold one copy of their body, without which it took two to three times
// as long.
//
// Units are shared out evenly over the CTAs by their tiles of 128 tokens (a unit's start and end
// count as kUnitCost more), whatever the lengths: a CTA's share may begin and end inside a unit, whose
// parts are then joined, in CTA order, by a second kernel.  Where few units of few tiles can have a CTA each, they
// get one, and there is nothing to join.
#include <cfloat>

#include "common.cuh"
#include "f8_convert.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kTileRows = 128, kUnitRows = 2 * kTileRows;
constexpr int kTok = 128;   // tokens of a tile
constexpr int kGroups = 8;  // of 16 tokens: the smallest block, and the K of one instruction
constexpr int kThreads = 512;
constexpr int kConvWarp = 8, kMmaWarp = 12, kPlanWarp = 13, kScoutWarp = 14, kLoadWarp = 15;
// 512 threads are launched with 128 registers each: 512 for the four warps of a sub-partition
// (184, 64 and 80 left values of the softmax's loop in local memory: 3 % slower)
constexpr uint32_t kSoftRegs = 208, kConvRegs = 48, kLowRegs = 48;
static_assert(2 * kSoftRegs + kConvRegs + kLowRegs <= 512, "register split");
constexpr int kStages = 2;  // of keys and of values
constexpr int kTabs = 8;    // tiles of which it is known where they lie
constexpr int kRing = 4;    // units
constexpr int kUnitCost = 3;  // what a unit's start and end cost, in tiles
constexpr int kMinShare = 4;  // tiles of a CTA's share, at least
constexpr float kLift = 5.f, kMost = 15.f, kMostP = 32768.f;  // (FP16 ends below 2^16)
constexpr uint32_t kSCol = 0, kOCol = 256;  // TMEM columns: S of tile i at 128 i, O at 256 + 128 i

// A part of a unit: tokens 128 j0 .. 128 j1 - 1 of what its rows see.
enum { kEnd = -1, kWhole = 0, kLater = 1, kFirst = 2 };  // kLater, kFirst: which of the CTA's two slots
struct Unit {
  int kind;
  int head, b;
  int t0, n;        // the sequence's new tokens
  int len;          // its tokens
  int row0, rows;   // rows of the sequence: token * group + query head
  int j0, j1;
  int first, vis;   // tokens that its first row and its last one see
  int bad;          // values that are not finite were hidden in tiles that some rows do not see whole
};

// What the join has to know of a unit that CTA c begins and others go on with.
struct Split {
  int parts;  // 0: none
  int head, t0, row0, rows;
};

// What the roles need of a tile of tokens, found ahead of them.
struct Scales {   // of 16 tokens
  float k;        // of the keys
  float add;      // log2 |v_scale| (or of kNoScale), -infinity without a block
  float inv;      // 1 / |v_scale|
  uint32_t mode;  // what becomes of the values' codes: see kZero, kNegate, kNotFinite
};
struct Tab {
  Scales g[kGroups];
  int row[kGroups];  // of the cache's rows [num_blocks, heads, block]: where 16 tokens begin, -1: nowhere
  int slot;          // the tile's unit; -1: no more tiles
  int all;           // all of them lie somewhere
  int last;          // of its unit
  int there, whole;  // tokens that the unit's last row sees, and its first one (may lie outside 0 .. 128)
  float v0;          // |v_scale| of its first tokens
  int pad[2];
};
// What stands for the |v_scale| of a block whose own is 0, below FP32's normal numbers or not finite: its tokens count in the
// weights' sum alone, so it is small, for the reference to be that of the blocks that reach the output (scales that
// fp8_kv_append makes of values down to 10^-15 are larger), and far enough from FP32's least for the sum to keep them.
constexpr float kNoScale = 0x1p-60f;
static_assert(sizeof(Tab) == 192, "tile record");
enum : uint32_t { kZero = 1, kNegate = 2, kNotFinite = 4 };

// Tokens that row r of a sequence sees.
__device__ __forceinline__ int row_limit(const KvChunkArgs& a, int len, int n, int r) {
  return a.causal ? max(0, len - n + 1 + r / a.group) : len;
}
__device__ __forceinline__ int unit_tiles(const KvChunkArgs& a, int len, int n, int u) {
  const int last = min(n * a.group, (u + 1) * kUnitRows) - 1;
  return (row_limit(a, len, n, last) + kTok - 1) / kTok;
}

// What unit u of a sequence counts for in the shares.
__device__ __forceinline__ int unit_cost(const KvChunkArgs& a, int len, int n, int u) {
  return a.whole ? 1 : unit_tiles(a, len, n, u) + kUnitCost;
}

struct Seq {
  int t0, n, len;
};
// Sequence b; n = 0 where its offsets are out of order, len = 0 where its length is.
__device__ __forceinline__ Seq sequence(const KvChunkArgs& a, int b, int* status) {
  Seq s = {0, 0, 0};
  if (b >= a.B) return s;
  bool ok = sequence_tokens(a.cu, b, a.B, a.T, a.max_q, &s.t0, &s.n);
  if (!ok) s.n = 0;
  s.len = a.lens[b];
  if (s.len < 0 || (long long)s.len > (long long)a.width * a.block) {
    s.len = 0;
    ok = false;
  }
  if (!ok) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
  return s;
}
__device__ __forceinline__ int units_of(const KvChunkArgs& a, int n) {
  return (n * a.group + kUnitRows - 1) / kUnitRows;
}

__device__ __forceinline__ long long shfl_up_ll(long long v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// What the units of the lane's sequence cost together; called by whole warps.
__device__ __forceinline__ long long sequence_cost(const KvChunkArgs& a, const Seq& s, int lane) {
  const int units = units_of(a, s.n);
  long long w = 0;
  if (units <= 4)
    for (int u = 0; u < units; ++u) w += unit_cost(a, s.len, s.n, u);
  uint32_t many = __ballot_sync(0xffffffffu, units > 4);
  while (many) {  // the lanes share a long sequence's
    const int l = __ffs(many) - 1;
    many &= many - 1;
    const int n = __shfl_sync(0xffffffffu, s.n, l), len = __shfl_sync(0xffffffffu, s.len, l);
    long long sum = 0;
    for (int u = lane; u < units_of(a, n); u += 32) sum += unit_cost(a, len, n, u);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == l) w = sum;
  }
  return w;
}

// The CTA's share of the work: [lo, hi) of the heads' lists of units, one list after the other.
struct Share {
  long long lo, hi, total, each;  // each: a CTA's share (the last one's may be less)
  int head, b;                    // where it begins: head, sequence, and cost of the sequence's units before
  long long off;
};

// a / b of numbers that are not negative; in 32 bits where they fit (code that runs once is slow by its length).
__device__ __forceinline__ long long quotient_ll(long long a, long long b) {
  if (((a | b) >> 32) == 0) return uint32_t(a) / uint32_t(b);
  return (unsigned long long)a / (unsigned long long)b;
}

// Share of a CTA when all heads' lists together cost heads * list.
__device__ __forceinline__ Share share_of(const KvChunkArgs& a, long long list) {
  Share sh;
  sh.total = list * a.heads;
  sh.each = max(a.whole ? 1LL : (long long)kMinShare, quotient_ll(sh.total + gridDim.x - 1, gridDim.x));
  sh.lo = min(sh.total, sh.each * blockIdx.x);
  sh.hi = min(sh.total, sh.lo + sh.each);
  sh.head = list > 0 ? int(quotient_ll(sh.lo, list)) : 0;
  sh.b = 0;
  sh.off = 0;
  return sh;
}

// Up to 32 sequences: one warp finds the share, and the sequence that it begins in, by itself, a lane each (the
// block's way took 1 us longer).
constexpr int kFew = 32;
__device__ __forceinline__ void find_share_few(const KvChunkArgs& a, int lane, Share* out, Seq* s, int* status) {
  const Seq mine = sequence(a, lane, status);
  const long long w = sequence_cost(a, mine, lane);
  long long upto = w;
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = shfl_up_ll(upto, o);
    if (lane >= o) upto += v;
  }
  const long long list = __shfl_sync(0xffffffffu, upto, 31);
  Share sh = share_of(a, list);
  const long long at = sh.lo - sh.head * list;
  const uint32_t in = __ballot_sync(0xffffffffu, at >= upto - w && at < upto);
  if (lane == (in ? __ffs(in) - 1 : 0)) {
    sh.b = lane;
    sh.off = at - (upto - w);
    *out = sh;
    *s = mine;
  }
  __syncwarp();
}

__device__ void find_share(const KvChunkArgs& a, Share* out, long long* sums, int* status) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  long long list = 0;
  Seq s = {0, 0, 0};
  long long w = 0, upto = 0;  // the thread's sequence and the cost up to its end (last round)
  int base = 0;
  // one round of 512 sequences: costs and their running sum
  auto round = [&]() {
    s = sequence(a, base + tid, status);
    w = sequence_cost(a, s, lane);
    upto = w;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = shfl_up_ll(upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long all = 0;
#pragma unroll 1
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) upto += sums[i];
      all += sums[i];
    }
    __syncthreads();
    return all;
  };
  for (base = 0; base < a.B; base += kThreads) list += round();
  const Share sh = share_of(a, list);
  if (tid == 0) *out = sh;
  __syncthreads();
  if (sh.lo >= sh.hi) return;
  const long long at = sh.lo - sh.head * list;
  long long before = 0;
  for (base = 0; base < a.B; base += kThreads) {
    const long long all = a.B > kThreads ? round() : list;  // (one round: the first one's are still there)
    if (at < before + all) {
      if (at >= before + upto - w && at < before + upto) {
        out->b = base + tid;
        out->off = at - (before + upto - w);
      }
      break;
    }
    before += all;
  }
  __syncthreads();
}

template <int kDim>
struct Smem {
  static constexpr int kTileBytes = kTok * kDim * 2;         // 128 rows of FP16
  static constexpr int kSubBytes = kTok * 128;
  static constexpr size_t kQ = 0, kK = kQ + 2 * kTileBytes, kV = kK + kStages * kTileBytes;
  static constexpr size_t kCodes = kV + kStages * kTileBytes;  // keys' and values' codes on their way
  static constexpr size_t kTab = kCodes + 2 * kTok * kDim;
  static constexpr size_t kUnits = kTab + kTabs * sizeof(Tab);
  static constexpr size_t kBars = kUnits + kRing * 64;
  static constexpr size_t kBytes = kBars + 512;
  static_assert(sizeof(Unit) <= 64, "ring slot");
  static_assert(kBytes <= 232448, "227 KB of shared memory per CTA");
};

struct Bars {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t tab_full[kTabs], tab_empty[kTabs];
  uint64_t codes_full[2], codes_empty[2];  // keys', values'
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  Share share;
  Seq seq;  // that it begins in
};
static_assert(sizeof(Bars) <= 512, "barrier area");

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16-byte chunk c of a row of the 64-element tiles that make up one of FP16.
template <int kDim>
__device__ __forceinline__ uint8_t* chunk_at(uint8_t* tile, int row, int c) {
  return tile + (c / 8) * Smem<kDim>::kSubBytes + row * 128 + (((c % 8) ^ (row & 7)) << 4);
}

// A warp's 32 rows of Q are asked for as they lie (`at`: where the lane's row begins, < 0: no such row;
// whole rows are read by neighbouring lanes) and become FP16 in place, times a power of two for each that
// brings its largest element into [2^10, 2^11): stage_queries returns the reciprocal of that power for the
// lane's row, the `row`-th of the tile.  (Code that runs once a unit is kept short too: it comes from
// beyond the instruction cache each time.)
template <int kDim>
__device__ __forceinline__ void request_queries(uint8_t* tile, int row, int lane, const __nv_bfloat16* Q, long long at) {
  constexpr int kChunks = kDim / 8, kRowsAtOnce = 32 / kChunks;
#pragma unroll 2
  for (int y = 0; y < 32; y += kRowsAtOnce) {
    const int from = y + lane / kChunks;
    const long long q = __shfl_sync(0xffffffffu, at, from);
    cp_async_16(smem_addr(chunk_at<kDim>(tile, row - lane + from, lane % kChunks)),
                Q + (q < 0 ? 0 : q + 8 * (lane % kChunks)), q < 0 ? 0u : 16u);
  }
}
template <int kDim>
__device__ __forceinline__ float stage_queries(uint8_t* tile, int row) {
  constexpr int kChunks = kDim / 8;
  cp_async_wait_all();
  __syncwarp();
  uint32_t top2 = 0u;  // of the even elements and of the odd ones: magnitudes of BF16 order as whole numbers do
#pragma unroll 2
  for (int c = 0; c < kChunks; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(chunk_at<kDim>(tile, row, c));
    top2 = __vmaxu2(__vmaxu2(__vmaxu2(top2, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu)),
                    v.w & 0x7fff7fffu);
  }
  const uint32_t top = max(top2 >> 16, top2 & 0xffffu);
  // rows below 2^-115 (zeros among them) take the largest shift whose reciprocal is a normal number: theirs and BF16's
  // subnormal numbers become normal ones
  const int exp = max(int(top >> 7), 11);
  const float up = __uint_as_float(uint32_t(264 - exp) << 23);  // 2^(10 - (exp - 127))
#pragma unroll 2
  for (int c = 0; c < kChunks; ++c) {
    uint4* p = reinterpret_cast<uint4*>(chunk_at<kDim>(tile, row, c));
    float f[8];
    unpack8(Raw8<__nv_bfloat16>{*p}, f);
    *p = make_uint4(f16x2_bits(f[0] * up, f[1] * up), f16x2_bits(f[2] * up, f[3] * up),
                    f16x2_bits(f[4] * up, f[5] * up), f16x2_bits(f[6] * up, f[7] * up));
  }
  return __uint_as_float(uint32_t(exp - 10) << 23);
}

// Piece y of lane x of four becomes piece x of lane y, after kBit = 1 and 2.
template <int kBit>
__device__ __forceinline__ void exchange(uint4 (&w)[4], int lane) {
  const bool high = lane & kBit;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint4& lo = w[kBit == 1 ? 2 * p : p];
    uint4& hi = w[kBit == 1 ? 2 * p + 1 : p + 2];
    uint4 send = high ? lo : hi;
    send.x = __shfl_xor_sync(0xffffffffu, send.x, kBit);
    send.y = __shfl_xor_sync(0xffffffffu, send.y, kBit);
    send.z = __shfl_xor_sync(0xffffffffu, send.z, kBit);
    send.w = __shfl_xor_sync(0xffffffffu, send.w, kBit);
    if (high)
      lo = send;
    else
      hi = send;
  }
}

// Bits of the bytes of a word that are no finite number (0xff in each).
template <bool kE5M2>
__device__ __forceinline__ uint32_t not_finite4(uint32_t w) {
  constexpr uint32_t kBad = kE5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
  return __vcmpeq4(w & kBad, kBad);
}

// The same value, of which the compiler knows nothing any more: it then makes no second copy of a loop's body
// for the first pass.
__device__ __forceinline__ bool opaque(bool b) {
  int x = b;
  asm volatile("" : "+r"(x));
  return x != 0;
}

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Block of token tok of the unit's sequence, -1 where there is none.
__device__ __forceinline__ int block_of(const KvChunkArgs& a, int b, int tok, int vis, int* status) {
  if (tok >= vis) return -1;
  const int blk = a.table[(long long)b * a.width + (tok >> a.log_block)];
  if (blk >= 0 && blk < a.num_blocks) return blk;
  raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
  return -1;
}

// Dimensions of tokens from .. to - 1 of which some value is not finite: bit d of `mask`.
template <int kDim, bool kE5M2>
__device__ __noinline__ void find_not_finite(const KvChunkArgs& a, int b, int head, int from, int to,
                                             int* status, uint32_t (&mask)[kDim / 32]) {
#pragma unroll 1
  for (int tok = from; tok < to; ++tok) {
    const int blk = block_of(a, b, tok, to, status);
    if (blk < 0) continue;
    const long long tile = (long long)blk * a.heads + head;
    const bool all = !(fabsf(a.vs[tile]) <= FLT_MAX);
    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.vc + (tile * a.block + (tok & (a.block - 1))) * kDim);
#pragma unroll
    for (int w = 0; w < kDim / 4; ++w) {
      const uint32_t m = all ? 0xffffffffu : not_finite4<kE5M2>(v[w]);
      // one bit of each byte, side by side
      mask[w / 8] |= ((m & 1u) | (m >> 7 & 2u) | (m >> 14 & 4u) | (m >> 21 & 8u)) << (w % 8 * 4);
    }
  }
}

template <int kDim, bool kE5M2>
__global__ void __launch_bounds__(kThreads, 1)
    kv_chunk_kernel(const __grid_constant__ KvChunkArgs a, float* parts, Split* splits, int* status) {
  using S = Smem<kDim>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (no static shared memory before it)
  Tab* tabs = reinterpret_cast<Tab*>(smem + S::kTab);
  auto ring = [&](int slot) { return reinterpret_cast<Unit*>(smem + S::kUnits + 64 * slot); };
  Bars& bar = *reinterpret_cast<Bars*>(smem + S::kBars);
  volatile int* abort_flag = &bar.abort;
  Share& share = bar.share;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.k_full[i], 4);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 4);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.codes_full[i], 1);
      mbar_init(&bar.codes_empty[i], 4);
      mbar_init(&bar.q_full[i], 4);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_full[i], 1);
    }
    for (int i = 0; i < kTabs; ++i) {
      mbar_init(&bar.tab_full[i], 1);
      mbar_init(&bar.tab_empty[i], 4);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&bar.ring_full[i], 1);
      mbar_init(&bar.ring_empty[i], 8 + 4 + 1);
    }
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  if (a.B > kFew) find_share(a, &share, reinterpret_cast<long long*>(smem), status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;

  auto fail = [&]() {
    *abort_flag = 1;
    raise_status(status, FP8GEMM_ERR_TIMEOUT);
  };
  // A whole warp's wait, with one outcome.  (Short: the roles' loops have to fit in the instruction
  // cache together.)
  auto warp_wait = [&](uint64_t* b, uint32_t parity, bool poll = false) {
    uint64_t t0 = 0;
    while (!__all_sync(0xffffffffu, poll ? mbar_test(b, parity) : mbar_try_wait(b, parity))) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, *abort_flag != 0 || now - t0 > a.wait_ns)) {
        fail();
        return false;
      }
    }
    return true;
  };

  if (warp < kConvWarp) {
    // ------------------------------------------------------------ softmax
    regs_increase<kSoftRegs>();
    const int i = warp / 4;                  // the tile
    const int row = (warp % 4) * 32 + lane;  // of the tile: TMEM lane
    const uint32_t lanes = uint32_t((warp % 4) * 32) << 16;
    const uint32_t s_at = tmem + lanes + kSCol + 128 * i, o_at = tmem + lanes + kOCol + 128 * i;
    uint8_t* q_tile = smem + S::kQ + i * S::kTileBytes;
    // where the lane's row of a unit lies in Q
    auto query_at = [&](const Unit* u) -> long long {
      const int r = kTileRows * i + row, sr = u->row0 + r;
      if (r >= u->rows) return -1;
      return (long long)(u->t0 + sr / a.group) * a.ld_q + (long long)(u->head * a.group + sr % a.group) * kDim;
    };
    bool asked = false;  // for the next unit's queries
    uint32_t it = 0;     // tiles of tokens, as all roles count them
    uint32_t mine = 0;   // those in which this tile of rows took part
    for (uint32_t taken = 0;; ++taken) {
      const int slot = taken % kRing;
      if (!warp_wait(&bar.ring_full[slot], (taken / kRing) & 1)) break;
      const Unit* u = ring(slot);
      const int kind = u->kind, rows = u->rows, j0 = u->j0, j1 = u->j1;
      if (kind == kEnd) break;
      if (rows <= kTileRows * i) {  // no rows for this tile
        it += j1 - j0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.ring_empty[slot]);
        continue;
      }
      const int r = kTileRows * i + row;  // row of the unit
      const bool row_ok = r < rows;
      const int seq_row = u->row0 + r;
      const int limit = row_ok ? row_limit(a, u->len, u->n, seq_row) : 0x7fffffff;
      const int least = __shfl_sync(0xffffffffu, limit, 0);  // rows see more and more
      const int most_seen = __reduce_max_sync(0xffffffffu, row_ok ? limit : 0);  // by a row of the warp
      float ref = 0.f, sum = 0.f, vref = 1.f;  // sum: of p over vref's share of |v_scale|
      bool unset = true;
      if (j1 > j0) {
        if (!asked) request_queries<kDim>(q_tile, row, lane, a.Q, query_at(u));
        const float down = stage_queries<kDim>(q_tile, row);
        asked = false;
        const float q_mul = down * (a.scale * 1.44269504088896341f);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_full[i]);
        bool ok = true;
        for (int j = j0; j < j1; ++j, ++it, ++mine) {
          const Scales* tab = tabs[it % kTabs].g;
          // (in this order: a tile of rows that sat out a unit may be ahead of the scales' ring, but
          // its own scores are there only once the tile's record is)
          if (!(ok = warp_wait(&bar.s_full[i], mine & 1))) break;
          if (!(ok = warp_wait(&bar.tab_full[it % kTabs], (it / kTabs) & 1))) break;
          tc_fence_after();
          if (j + 1 == j1) {  // the unit's queries have been used: those of the next one, if it is known yet
            const int next = (taken + 1) % kRing;
            if (__all_sync(0xffffffffu, mbar_test(&bar.ring_full[next], ((taken + 1) / kRing) & 1))) {
              const Unit* v = ring(next);
              asked = v->kind != kEnd && v->rows > kTileRows * i && v->j1 > v->j0;
              if (asked) request_queries<kDim>(q_tile, row, lane, a.Q, query_at(v));
            }
          }
          const int tok = j * kTok;
          if (j == j0) vref = tabs[it % kTabs].v0;
          if (__any_sync(0xffffffffu, unset)) {  // a first reference, from the first tile that is there
            float top = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < kTok / 32; ++h) {
              uint32_t c[32];
              tmem_ld_32x32b_x32(s_at + 32 * h, c);
              tmem_ld_wait_tied(c);
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const float mul = q_mul * tab[2 * h + g].k, add = tab[2 * h + g].add;
#pragma unroll
                for (int e = 16 * g; e < 16 * g + 16; ++e) {
                  const float x = fmaf(__uint_as_float(c[e]), mul, add);
                  if (tok + 32 * h + e < limit) top = fmaxf(top, x);
                }
              }
            }
            if (unset && top > -INFINITY) {
              ref = top - kLift;  // the largest P a power of two, which FP16 holds exactly
              unset = false;
            }
          }
          // What has been summed so far shrinks as the reference rises.
          auto rescale = [&](float shrink) {
            sum *= shrink;
            if (j == j0 || !__any_sync(0xffffffffu, shrink != 1.f)) return true;
            if (!warp_wait(&bar.o_full[i], (mine - 1) & 1)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < kDim; d += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(o_at + d, o);
              tmem_ld_wait_tied16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
              tmem_st_32x32b_x16(o_at + d, o);
            }
            return true;
          };
          // The plain case, to which most tiles belong: all rows see all tokens.  That the reference need not rise
          // is known once P is there, in registers; if it has to, P is formed again.
          bool plain = !__any_sync(0xffffffffu, unset) && tok + kTok <= least;
#pragma unroll 1
          while (opaque(plain)) {
            uint32_t c[3][32], p[4][16];
            float part = 0.f, most = 0.f;
            auto take = [&](const uint32_t (&from)[32], int h) {  // 32 tokens
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const float mul = q_mul * tab[2 * h + g].k, add = tab[2 * h + g].add - ref;
                float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const float2 x =
                      __ffma2_rn(make_float2(__uint_as_float(from[16 * g + e]), __uint_as_float(from[16 * g + e + 1])),
                                 make_float2(mul, mul), make_float2(add, add));
                  const float2 v = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                  sum2 = __fadd2_rn(sum2, v);
                  p[h][8 * g + e / 2] = f16x2_bits(v.x, v.y);
                }
                const float sum1 = sum2.x + sum2.y;
                most = fmaxf(most, sum1);  // no P is larger
                part = fmaf(sum1, tab[2 * h + g].inv * vref, part);
              }
            };
            // two loads ahead: they take long beside the products' own traffic
            tmem_ld_32x32b_x32(s_at, c[0]);
            tmem_ld_32x32b_x32(s_at + 32, c[1]);
            tmem_ld_wait_tied(c[0]);
            reg_tie32(c[1]);
            tmem_ld_32x32b_x32(s_at + 64, c[2]);
            take(c[0], 0);
            tmem_ld_32x32b_x32(s_at + 96, c[0]);
            take(c[1], 1);
            tmem_ld_wait_tied(c[2]);
            reg_tie32(c[0]);
            take(c[2], 2);
            take(c[0], 3);
            if (!__any_sync(0xffffffffu, most > kMostP)) {
              sum += part;
#pragma unroll
              for (int h = 0; h < 4; ++h) tmem_st_32x32b_x16(s_at + 16 * h, p[h]);
              break;
            }
            // (`most` is up to 16 times the largest P.  What it cannot tell goes the other way: infinity, and
            // references so large that they hardly rise.)
            float up = 0.f;
            if (most > kMostP) up = float(int(__float_as_uint(most) >> 23) - 127) - kLift;
            const float to = ref + up;
            plain = !__any_sync(0xffffffffu, most == INFINITY || !(to - ref > up - 1.f));
            if (plain) {
              up = to - ref;
              ref = to;
              if (!(ok = rescale(exp2_fast(-up)))) break;
            }
          }
          if (!ok) break;
#pragma unroll 1
          for (int h = plain ? kTok / 32 : 0; h < kTok / 32; ++h) {  // 32 tokens at a time
            const int sees = limit - tok - 32 * h;
            uint32_t p[16];
            float sums[2];
            if (tok + 32 * h >= most_seen) {  // no row sees any of these
#pragma unroll
              for (int e = 0; e < 16; ++e) p[e] = 0u;
              tmem_st_32x32b_x16(s_at + 16 * h, p);
              continue;
            }
            // Once as if the reference need not rise; if it has to, again with the new one.
#pragma unroll 1
            for (bool again = opaque(false);; again = opaque(true)) {
              uint32_t c[32];
              tmem_ld_32x32b_x32(s_at + 32 * h, c);
              tmem_ld_wait_tied(c);
              float x[32];  // scores in powers of two, with the value scale's, less the reference
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[e] = fmaf(__uint_as_float(c[e]), q_mul * tab[2 * h + e / 16].k, tab[2 * h + e / 16].add - ref);
              if (tok + 32 * h + 32 > least) {  // the same for the warp: some row does not see all of these
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e >= sees) x[e] = -INFINITY;
              }
              if (again) {  // scores of 2^27 and more: a rounded reference may lie far below the largest
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = min_nan(x[e], kLift + 1.f);
              }
              float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                float sum_a = 0.f, sum_b = 0.f;
#pragma unroll
                for (int e = 16 * g; e < 16 * g + 16; e += 2) {
                  if (e % 4)
                    top1 = max3(top1, x[e], x[e + 1]);
                  else
                    top0 = max3(top0, x[e], x[e + 1]);
                  const float va = exp2_fast(x[e]), vb = exp2_fast(x[e + 1]);
                  sum_a += va;
                  sum_b += vb;
                  p[e / 2] = f16x2_bits(va, vb);
                }
                sums[g] = sum_a + sum_b;
              }
              const float top = fmaxf(top0, top1);
              if (again || !__any_sync(0xffffffffu, top > kMost)) break;
              // by how much the reference rises: a whole number, for what is there to be multiplied by a power of two
              const float to = ref + floorf(fmaxf(top - kLift, 0.f));
              const float shrink = exp2_fast(ref - to);
              ref = to;
              // P of the tile's tokens before these, in FP32: exact but for what FP16 then holds with fewer bits
              if (h > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
                tmem_st_wait();
#pragma unroll 1
                for (int d = 0; d < 16 * h; d += 16) {
                  uint32_t o[16];
                  tmem_ld_32x32b_x16(s_at + d, o);
                  tmem_ld_wait_tied16(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
                    o[e] = f16x2_bits(v.x * shrink, v.y * shrink);
                  }
                  tmem_st_32x32b_x16(s_at + d, o);
                }
              }
              if (!(ok = rescale(shrink))) break;
            }
            if (!ok) break;
#pragma unroll
            for (int g = 0; g < 2; ++g) sum = fmaf(sums[g], tab[2 * h + g].inv * vref, sum);
            tmem_st_32x32b_x16(s_at + 16 * h, p);  // (where scores have been used)
          }
          if (!ok) break;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full[i]);
        }
        if (!ok || !warp_wait(&bar.o_full[i], (mine - 1) & 1)) break;
        tc_fence_after();
      }
      // ---- the rows' end: whole units go to O, parts to the workspace
      if (u->bad) {  // such rows' O becomes NaN where they see a value that is not finite
        uint32_t lost[kDim / 32] = {};
        if (row_ok)
          find_not_finite<kDim, kE5M2>(a, u->b, u->head, max(u->first / kTok * kTok, j0 * kTok), min(limit, j1 * kTok),
                                       status, lost);
        __syncwarp();
#pragma unroll 1
        for (int d = 0; d < kDim; d += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(o_at + d, o);
          tmem_ld_wait_tied(o);
          const uint32_t m = lost[d / 32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (m >> e & 1u) o[e] = 0x7fc00000u;
          tmem_st_32x32b_x32(o_at + d, o);
        }
        tmem_st_wait();
      }
      // (times vref first, whose share is in the sum: the product is about a value scale)
      const float f = (sum > 0.f || isnan(sum) ? __fdividef(1.f, sum) : 0.f) * vref;
      const long long out = !row_ok ? -1 : ((long long)(u->t0 + seq_row / a.group) * a.heads * a.group +
                                      u->head * a.group + seq_row % a.group) * kDim;
      // parts: [kDim / 4][rows][4], then [rows][4], so that neighbouring lanes write neighbouring places
      float4* part = reinterpret_cast<float4*>(parts) +
                     (size_t(blockIdx.x) * 2 + (kind == kFirst)) * (kUnitRows * (kDim / 4 + 1)) + r;
#pragma unroll 1
      for (int d = 0; d < kDim; d += 32) {
        uint32_t o[32] = {};
        if (j1 > j0) {
          tmem_ld_32x32b_x32(o_at + d, o);
          tmem_ld_wait_tied(o);
        }
        if (kind == kWhole) {
          // four lanes exchange their rows' pieces so that they write 64 bytes of a row together (16 bytes a
          // row from each lane took as long as the rest of a unit's end)
          uint4 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) v[y] = __uint_as_float(o[8 * e + y]) * f;
            w[e] = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
          }
          exchange<1>(w, lane);
          exchange<2>(w, lane);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const long long at = __shfl_sync(0xffffffffu, out, (lane & ~3) + y);
            if (at >= 0) *reinterpret_cast<uint4*>(a.O + at + d + 8 * (lane & 3)) = w[y];
          }
        } else if (row_ok) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            part[size_t(d + e) / 4 * kUnitRows] =
                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                            __uint_as_float(o[e + 3]));
        }
        __syncwarp();
      }
      if (kind != kWhole && row_ok) {
        part[size_t(kUnitRows) * (kDim / 4)] = make_float4(unset ? -INFINITY : ref, sum, vref, 0.f);
      }
      tc_fence_before();  // O has been read before its next product, which waits for P
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ring_empty[slot]);
    }
    cp_async_wait_all();
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------- keys and values
    regs_decrease<kConvRegs>();
    const int ct = threadIdx.x - 32 * kConvWarp;
    // Eight neighbouring threads have the eight (four) pieces of two neighbouring tokens such that both the
    // codes and the chunks of FP16 that they become meet all banks.
    const int piece = kDim == 128 ? ct & 7 : ct & 3;
    const int row0 = kDim == 128 ? ct >> 3 ^ (piece >> 2) : ct >> 2;
    constexpr int kRowsAtOnce = 128 / (kDim / 16);  // tokens that the 128 threads cover at once: a multiple of 8
    constexpr int kLoads = kTok / kRowsAtOnce;
    const uint32_t to0 = uint32_t(chunk_at<kDim>(smem, row0, 2 * piece) - smem);
    const uint32_t to1 = uint32_t(chunk_at<kDim>(smem, row0, 2 * piece + 1) - smem);
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int st = it % kStages;
      const uint32_t ph = (it / kStages) & 1;
      const Tab& tab = tabs[it % kTabs];
      if (!warp_wait(&bar.tab_full[it % kTabs], (it / kTabs) & 1) || tab.slot < 0) break;
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {  // keys, values
        uint8_t* codes = smem + S::kCodes + v * kTok * kDim + row0 * kDim + 16 * piece;
        if (!(ok = warp_wait(v ? &bar.v_empty[st] : &bar.k_empty[st], ph ^ 1))) break;
        // the values of two tiles ago have been used, and so have their scales
        if (v == 1 && lane == 0 && it >= 2) mbar_arrive(&bar.tab_empty[(it - 2) % kTabs]);
        if (!(ok = warp_wait(&bar.codes_full[v], it & 1))) break;
        const bool mixed = tab.whole < kTok;
        if (!tab.all || (v == 1 && __any_sync(0xffffffffu, mixed || tab.g[lane % kGroups].mode != 0u))) {
          // Tokens without a block: nothing was copied to their places.  Or some value scale is 0, negative or not
          // finite, or some row does not see the whole tile.  There 0 times what is not finite would
          // reach rows that do not see it: such values become 0, and the rows that do see them are
          // marked when the unit ends.
          uint32_t bad = 0u;
#pragma unroll 2
          for (int l = 0; l < kLoads; ++l) {
            const int r = row0 + kRowsAtOnce * l;
            const uint32_t mode = v == 1 ? tab.g[r / 16].mode : 0u;
            uint4* at = reinterpret_cast<uint4*>(codes + l * kRowsAtOnce * kDim);
            const uint4 x = *at;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            // Bits of a code: those that are there, those whose value a scale of 0 leaves, those to be looked at, all of
            // a scale that is not finite.
            const uint32_t there = tab.row[r / 16] < 0 || r >= tab.there ? 0u : 0xffffffffu;
            const uint32_t kept = mode & kZero ? 0u : there;
            const uint32_t seen = (mixed && v == 1) || mode & kZero ? there : 0u;
            const uint32_t all = mode & kNotFinite ? there : 0u;
            const uint32_t sign = mode & kNegate ? 0x80808080u : 0u;
            const uint32_t nan = mixed ? 0u : 0x7f7f7f7fu;  // in either format
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lost = (not_finite4<kE5M2>(w[e]) & seen) | all;  // (0 times what is not finite is NaN)
              bad |= lost;
              w[e] = (((w[e] ^ sign) & kept) & ~lost) | (lost & nan);
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (mixed && bad) ring(tab.slot)->bad = 1;
        }
        uint8_t* tile = smem + (v ? S::kV : S::kK) + st * S::kTileBytes;
#pragma unroll 1
        for (int l0 = 0; l0 < kLoads; l0 += 4) {
          uint4 x[4];
#pragma unroll
          for (int l = 0; l < 4; ++l) x[l] = *reinterpret_cast<const uint4*>(codes + (l0 + l) * kRowsAtOnce * kDim);
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            const uint32_t w[4] = {x[l].x, x[l].y, x[l].z, x[l].w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[2 * e] = f8x2_to_f16x2<kE5M2>(uint16_t(w[e]));
              y[2 * e + 1] = f8x2_to_f16x2<kE5M2>(uint16_t(w[e] >> 16));
            }
            const int at = (l0 + l) * kRowsAtOnce * 128;
            *reinterpret_cast<uint4*>(tile + to0 + at) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(tile + to1 + at) = make_uint4(y[4], y[5], y[6], y[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v ? &bar.v_full[st] : &bar.k_full[st]);
          mbar_arrive(&bar.codes_empty[v]);
        }
      }
      if (ok && tab.last && lane == 0) mbar_arrive(&bar.ring_empty[tab.slot]);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------- the products
    // The whole warp runs this, in step, so that descriptors stay in uniform registers; one lane issues.
    regs_decrease<kLowRegs>();
    constexpr uint32_t kDescS = idesc_f16_f32(kTileRows, kTok, false);
    constexpr uint32_t kDescO = idesc_f16_f32(kTileRows, kDim, true);
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
    const uint64_t q_desc = smem_desc_sw128_kmajor(smem_addr(smem + S::kQ));
    const uint64_t k_desc = smem_desc_sw128_kmajor(smem_addr(smem + S::kK));
    const uint64_t v_desc = smem_desc_sw128_mnmajor(smem_addr(smem + S::kV), S::kSubBytes);
    uint32_t it = 0, n_0 = 0, n_1 = 0, units_0 = 0, units_1 = 0;
    bool issued = false;
    auto scores = [&](int i, int st) {
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kDim / 16; ++k) {
          const uint32_t off = ((k / 4) * S::kSubBytes + (k % 4) * 32) >> 4;
          umma_f16(tm + kSCol + 128 * i, q_desc + (off + i * (S::kTileBytes >> 4)),
                   k_desc + (off + st * (S::kTileBytes >> 4)), kDescS, k > 0 ? 1u : 0u);
        }
        umma_commit(&bar.s_full[i]);
      }
      issued = true;
    };
    auto values = [&](int i, int st, bool first) {
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTok / 16; ++k)
          umma_f16_ta(tm + kOCol + 128 * i, tm + kSCol + 128 * i + 8 * k,
                      v_desc + (k * (2048 >> 4) + st * (S::kTileBytes >> 4)), kDescO, first && k == 0 ? 0u : 1u);
        umma_commit(&bar.o_full[i]);
      }
    };
    auto commit = [&](uint64_t* b) {
      if (elect_one()) umma_commit(b);
    };
    bool ok = true;
    for (uint32_t taken = 0; ok; ++taken) {
      const int slot = taken % kRing;
      if (!warp_wait(&bar.ring_full[slot], (taken / kRing) & 1)) break;
      const Unit* u = ring(slot);
      const int n = __reduce_max_sync(0xffffffffu, u->kind == kEnd ? -1 : u->j1 - u->j0);
      const int tiles = __reduce_max_sync(0xffffffffu, u->rows > kTileRows ? 2 : 1);
      if (n < 0) break;
#pragma unroll 1
      for (int j = 0; j <= n && n > 0; ++j) {  // scores of tile j behind the values of tile j - 1
        const uint32_t before = it - 1;
        if (j < n) ok = warp_wait(&bar.k_full[it % kStages], (it / kStages) & 1);
        if (ok && j > 0) ok = warp_wait(&bar.v_full[before % kStages], (before / kStages) & 1);
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
          const uint32_t n_i = i ? n_1 : n_0;  // tiles of tokens that this tile of rows has had
          if (j == 0)
            ok = warp_wait(&bar.q_full[i], (i ? units_1++ : units_0++) & 1);
          else
            ok = warp_wait(&bar.p_full[i], (n_i + j - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (j > 0) values(i, before % kStages, j == 1);
          if (j < n) scores(i, it % kStages);
        }
        if (!ok) break;
        if (j > 0) commit(&bar.v_empty[before % kStages]);
        if (j < n) {
          commit(&bar.k_empty[it % kStages]);
          ++it;
        }
      }
      n_0 += n;
      if (tiles > 1) n_1 += n;
      if (ok && lane == 0) mbar_arrive(&bar.ring_empty[slot]);
    }
    if (issued) {  // every issued product has finished before TMEM is released
      commit(&bar.drain);
      mbar_drain(&bar.drain, 0);
    }
  } else {
    regs_decrease<kLowRegs>();
    if (warp == kPlanWarp) {
      // ------------------------------------------------- units of the CTA's share
      Split split = {0, 0, 0, 0, 0};
      uint32_t given = 0;
      bool ok = true;
      auto give = [&](const Unit& unit) {
        const int slot = given % kRing;
        if (!warp_wait(&bar.ring_empty[slot], ((given / kRing) & 1) ^ 1)) return false;
        if (lane == 0) {
          *ring(slot) = unit;
          mbar_arrive(&bar.ring_full[slot]);
        }
        ++given;
        return true;
      };
      if (a.B <= kFew) find_share_few(a, lane, &share, &bar.seq, status);
      Seq s = bar.seq;
      if (a.B > kFew) s = sequence(a, share.b, status);
      const long long lo = share.lo, hi = share.hi;
      if (lo < hi) {
        long long at = lo, off = share.off;  // off: cost before `at` within the sequence, then the unit
        int head = share.head, b = share.b, un = 0;
        // the unit that holds the offset, 32 at a time
        while (true) {
          const int u = un + lane;
          const int w = u < units_of(a, s.n) ? unit_cost(a, s.len, s.n, u) : 0;
          int upto = w;
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, off < upto);
          if (past) {
            const int l = __ffs(past) - 1;
            off -= __shfl_sync(0xffffffffu, upto - w, l);
            un += l;
            break;
          }
          off -= __shfl_sync(0xffffffffu, upto, 31);
          un += 32;
          if (un >= units_of(a, s.n)) break;  // (cannot be: the offset lies in the sequence)
        }
        while (at < hi && ok) {
          while (un >= units_of(a, s.n)) {  // on to the next sequence that has tokens, or the next head's list
            un = 0;
            const Seq next = sequence(a, b + 1 + lane, status);  // (none behind the last)
            const uint32_t some = __ballot_sync(0xffffffffu, next.n > 0);
            const int l = some ? __ffs(some) - 1 : 31;
            s.t0 = __shfl_sync(0xffffffffu, next.t0, l);
            s.n = __shfl_sync(0xffffffffu, next.n, l);
            s.len = __shfl_sync(0xffffffffu, next.len, l);
            b += 1 + l;
            if (b >= a.B) {
              b = -1;
              s.n = 0;
              ++head;
            }
          }
          const int tiles = unit_tiles(a, s.len, s.n, un);
          const long long cost = unit_cost(a, s.len, s.n, un), begin = at - off;
          const long long x1 = min(cost, off + (hi - at));
          Unit unit;
          unit.head = head;
          unit.b = b;
          unit.t0 = s.t0;
          unit.n = s.n;
          unit.len = s.len;
          unit.row0 = un * kUnitRows;
          unit.rows = min(kUnitRows, s.n * a.group - unit.row0);
          unit.j0 = int(max(0LL, off - kUnitCost));
          unit.j1 = a.whole ? tiles : int(max(0LL, x1 - kUnitCost));
          unit.first = row_limit(a, s.len, s.n, unit.row0);
          unit.vis = row_limit(a, s.len, s.n, unit.row0 + unit.rows - 1);
          unit.bad = 0;
          unit.kind = unit.j0 > 0 ? kLater : unit.j1 < tiles ? kFirst : kWhole;
          if (tiles == 0 ? off == 0 : unit.j1 > unit.j0) {
            if (unit.kind == kFirst) {
              const long long end = begin + cost;  // its parts: this CTA's and those that begin before its end
              int last = blockIdx.x;
              while (share.each * (last + 1) < end) ++last;
              split = {last - int(blockIdx.x) + 1, head, s.t0, unit.row0, unit.rows};
            }
            ok = give(unit);
            const int t0 = unit.t0 + unit.row0 / a.group, t1 = unit.t0 + (unit.row0 + unit.rows - 1) / a.group;
            for (int t = t0 + lane; t <= t1 && a.group <= kUnitRows; t += 32)  // its queries (not all of a wider group's)
              prefetch_l2(a.Q + (long long)t * a.ld_q + (long long)head * a.group * kDim, a.group * kDim * 2);
          }
          at += x1 - off;
          off = 0;
          ++un;
        }
      }
      if (lane == 0) splits[blockIdx.x] = split;
      Unit end = {};
      end.kind = kEnd;
      if (ok) give(end);
    } else if (warp == kLoadWarp) {
      // ------------------------------------------- codes into shared memory, 16 tokens a copy
      constexpr uint32_t kBytes = 16 * kDim;
      // One try of a wait may sleep for many microseconds: limits under 100 us are kept by this warp, which polls for
      // them (all roles doing so took 0.5 % of the call's time).
      const bool poll = a.wait_ns < 100000;
      bool ok = true;
      uint32_t asked = 0;  // copies, keys' and values' in turn
      for (uint32_t it = 0; ok; ++it) {
        const Tab& tab = tabs[it % kTabs];
        if (!(ok = warp_wait(&bar.tab_full[it % kTabs], (it / kTabs) & 1, poll)) || tab.slot < 0) break;
        const int row = lane < kGroups ? tab.row[lane] : -1;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0));
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          if (!(ok = warp_wait(&bar.codes_empty[v], (it & 1) ^ 1, poll))) break;
          ++asked;
          if (lane == 0) mbar_arrive_expect_tx(&bar.codes_full[v], n * kBytes);
          __syncwarp();
          if (row >= 0)
            bulk_load(smem + S::kCodes + v * kTok * kDim + lane * kBytes, (v ? a.vc : a.kc) + (long long)row * kDim,
                      kBytes, &bar.codes_full[v]);
        }
      }
      // what is on its way lands before the CTA's end
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (asked > uint32_t(v)) mbar_drain(&bar.codes_full[v], ((asked - v + 1) / 2 - 1) & 1);
    } else if (warp == kScoutWarp) {
      // ------------------------------------------- where tiles lie, and their scales
      // Up to four tiles at a time, eight lanes each: table entries, then scales, are the latencies that nothing
      // else of the tile can start before.
      uint32_t it = 0, taken = 0;
      int j = 0, j1 = 0, slot = 0;
      bool ended = false, ok = true;
      while (ok && !ended) {
        int mine = -1, mine_j = 0;  // the lane's tile: its unit's slot
        int n = 0;
#pragma unroll 1
        for (; n < 4; ++n) {
          while (j == j1) {
            const int s = taken % kRing;
            const uint32_t ph = (taken / kRing) & 1;
            // what has been found is not held back for a unit that is not there yet
            if (n > 0 && !__all_sync(0xffffffffu, mbar_test(&bar.ring_full[s], ph))) break;
            if (!(ok = warp_wait(&bar.ring_full[s], ph))) break;
            const Unit* u = ring(s);
            if (u->kind == kEnd) {
              ended = true;
              break;
            }
            ++taken;
            slot = s;
            j = u->j0;
            j1 = u->j1;
            if (j == j1) {  // no tiles: the converters will not see it
              __syncwarp();
              if (lane < 4) mbar_arrive(&bar.ring_empty[s]);
            }
          }
          if (j == j1) break;
          if (lane / kGroups == n) {
            mine = slot;
            mine_j = j;
          }
          ++j;
        }
        if (!ok) break;
        const int g = lane % kGroups;
        const Unit* u = ring(max(mine, 0));
        const int tok = mine_j * kTok + 16 * g;
        const bool wanted = mine >= 0 && tok < u->vis;
        int blk = -1;
        if (wanted) {
          blk = a.table[(long long)u->b * a.width + (tok >> a.log_block)];
          if (blk < 0 || blk >= a.num_blocks) {
            raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
            blk = -1;
          }
        }
        float ks = 0.f, vs = 0.f;
        int row = -1;
        if (blk >= 0) {
          const int tile = blk * a.heads + u->head;  // (rows of the cache are fewer than 2^31)
          ks = a.ks[tile];
          vs = a.vs[tile];
          row = tile * a.block + (tok & (a.block - 1));
          prefetch_l2(a.kc + (long long)row * kDim, 16 * kDim);
          prefetch_l2(a.vc + (long long)row * kDim, 16 * kDim);
        }
        const bool fin = fabsf(vs) <= FLT_MAX, used = fin && fabsf(vs) >= FLT_MIN;
        const float av = used ? fabsf(vs) : kNoScale;
        Scales x;
        x.k = ks;
        // (its error is one of the weight of these tokens: 2^-15 at most)
        x.add = blk >= 0 ? __log2f(av) : -INFINITY;
        x.inv = blk >= 0 ? __frcp_rn(av) : 0.f;
        x.mode = blk < 0 ? kZero : !fin ? kNotFinite : !used ? kZero : vs < 0.f ? kNegate : 0u;
        const uint32_t lie = __ballot_sync(0xffffffffu, row >= 0);
        const int total = n + (ended ? 1 : 0);  // and the end
#pragma unroll 1
        for (int q = 0; q < total && ok; ++q, ++it) {
          Tab& t = tabs[it % kTabs];
          if (!(ok = warp_wait(&bar.tab_empty[it % kTabs], ((it / kTabs) & 1) ^ 1))) break;
          if (q == n) {
            if (lane == 0) t.slot = -1;
          } else if (lane / kGroups == q) {
            t.g[g] = x;
            t.row[g] = row;
            if (g == 0) {
              t.slot = mine;
              t.all = (lie >> (8 * q) & 0xffu) == 0xffu;
              t.last = mine_j + 1 == u->j1;
              t.there = u->vis - mine_j * kTok;
              t.whole = u->first - mine_j * kTok;
              t.v0 = av;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.tab_full[it % kTabs]);
        }
      }
    }
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the unit that CTA blockIdx.x of the kernel above began, in the order of the CTAs: a
// thread for each row, 16 dimensions a CTA.
constexpr int kJoinDims = 16;
template <int kDim>
__global__ void __launch_bounds__(kUnitRows) kv_chunk_join_kernel(const __grid_constant__ KvChunkArgs a,
                                                                  const float4* __restrict__ parts,
                                                                  const Split* __restrict__ splits) {
  griddep_launch_dependents();
  griddep_wait();
  const Split s = splits[blockIdx.x];
  const int r = threadIdx.x, d = blockIdx.y * kJoinDims;
  if (s.parts == 0 || r >= s.rows) return;
  constexpr size_t kSlot = size_t(kUnitRows) * (kDim / 4 + 1);
  auto part = [&](int p) { return parts + (size_t(blockIdx.x + p) * 2 + (p == 0)) * kSlot + r; };
  auto stat = [&](int p) { return part(p)[size_t(kUnitRows) * (kDim / 4)]; };
  // two parts at a time, statistics and rows asked for together
  float top = -INFINITY, sum = 0.f, vref = 1.f;
  float4 o[kJoinDims / 4] = {};
#pragma unroll 1
  for (int p = 0; p < s.parts; p += 2) {
    const bool two = p + 1 < s.parts;
    const int q = two ? p + 1 : p;
    const float4 t0 = stat(p), t1 = stat(q);
    float4 v0[kJoinDims / 4], v1[kJoinDims / 4];
#pragma unroll
    for (int i = 0; i < kJoinDims / 4; ++i) {
      v0[i] = part(p)[size_t(d / 4 + i) * kUnitRows];
      v1[i] = part(q)[size_t(d / 4 + i) * kUnitRows];
    }
    if (p == 0) vref = t0.z;
    const float up = max_nan(top, max_nan(t0.x, t1.x));
    const float shrink = top == -INFINITY ? 1.f : exp2_fast(top - up);  // (of nothing yet)
    const float w0 = t0.x == -INFINITY ? 0.f : exp2_fast(t0.x - up);
    const float w1 = !two || t1.x == -INFINITY ? 0.f : exp2_fast(t1.x - up);
    top = up;
    sum = fmaf(t1.y, w1 * __fdiv_rn(vref, t1.z), fmaf(t0.y, w0 * __fdiv_rn(vref, t0.z), sum * shrink));
#pragma unroll
    for (int i = 0; i < kJoinDims / 4; ++i) {
      o[i].x = fmaf(v1[i].x, w1, fmaf(v0[i].x, w0, o[i].x * shrink));
      o[i].y = fmaf(v1[i].y, w1, fmaf(v0[i].y, w0, o[i].y * shrink));
      o[i].z = fmaf(v1[i].z, w1, fmaf(v0[i].z, w0, o[i].z * shrink));
      o[i].w = fmaf(v1[i].w, w1, fmaf(v0[i].w, w0, o[i].w * shrink));
    }
  }
  const float f = (sum > 0.f || isnan(sum) ? __fdividef(1.f, sum) : 0.f) * vref;
  const int row = s.row0 + r;
  __nv_bfloat16* out =
      a.O + (((long long)s.t0 + row / a.group) * a.heads * a.group + s.head * a.group + row % a.group) * kDim + d;
  auto scaled = [&](float v) { return v * f; };
#pragma unroll
  for (int i = 0; i < kJoinDims / 4; i += 2)
    *reinterpret_cast<uint4*>(out + 4 * i) =
        make_uint4(bf16x2_bits(scaled(o[i].x), scaled(o[i].y)), bf16x2_bits(scaled(o[i].z), scaled(o[i].w)),
                   bf16x2_bits(scaled(o[i + 1].x), scaled(o[i + 1].y)), bf16x2_bits(scaled(o[i + 1].z), scaled(o[i + 1].w)));
}

// Units and tiles of a unit that a call has at most.
long long most_units(const KvChunkArgs& a) { return (long long)a.heads * ((long long)a.T * a.group / kUnitRows + a.B); }
long long most_tiles(const KvChunkArgs& a) { return ((long long)a.width * a.block + kTok - 1) / kTok; }

// Whole units, a CTA each, where sharing their tiles out cannot win what the join costs: tables of up to 4 tiles
// (17 tokens behind 37: 9.5 us, shared out 10.6; 512 x 64 heads 19.9 and 26.4), of up to 8 where units for half of
// the CTAs and more leave little to share out (1024 x 32 heads: 26.0 and 32.6; but 1024 x 2 heads 26.7 and 25.2, and
// 1964 tokens for 128 units 40 and 35).
bool whole_units(const LaunchCtx& c, const KvChunkArgs& a) {
  const long long units = most_units(a);
  return units <= c.num_sms && most_tiles(a) <= (2 * units >= c.num_sms ? 8 : 4);
}

template <int kDim, bool kE5M2>
cudaError_t run(const LaunchCtx& c, KvChunkArgs a, void* ws, int* launches) {
  static SmemLimit limit;
  auto fn = kv_chunk_kernel<kDim, kE5M2>;
  if (cudaError_t e = limit.raise(c, reinterpret_cast<const void*>(fn), Smem<kDim>::kBytes)) return e;
  // no more CTAs than there can be work for
  const long long units = most_units(a), tiles = most_tiles(a);
  a.whole = whole_units(c, a);
  const long long most = units > c.num_sms ? c.num_sms : a.whole ? units : units * (tiles + kUnitCost) / kMinShare;
  const int grid = int(min((long long)c.num_sms, max(1LL, most)));
  Split* splits = static_cast<Split*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(ws) + size_t(c.num_sms) * 64);
  if (cudaError_t e = launch_dependent(c, fn, grid, kThreads, Smem<kDim>::kBytes, a, parts, splits, c.status)) return e;
  *launches = 1;
  if (a.whole) return cudaSuccess;
  *launches = 2;
  return launch_dependent(c, kv_chunk_join_kernel<kDim>, dim3(grid, kDim / kJoinDims), kUnitRows, 0, a,
                          reinterpret_cast<const float4*>(parts), splits);
}

}  // namespace

// Two parts of a unit for each CTA, at dim 128: the same for every call, so that a stream's buffer stays
// where it is.
size_t kv_chunk_workspace_bytes(const LaunchCtx& c) {
  static_assert(sizeof(Split) <= 64, "split record");
  return size_t(c.num_sms) * (64 + 2 * size_t(kUnitRows) * (128 + 4) * 4);
}

// The cache attention for single tokens (16 rows of a cached head a pass, at the memory's rate) takes up to 32 rows
// faster (128 dimensions, 8 cached heads; us there / here: 8 rows over 100000 tokens 41 / 80, 64 sequences of 300 tokens with
// 16 rows 25 / 48, with 32 rows 38 / 48, 16 of 16000 with 32 rows 184 / 177, with 64 rows 339 / 178), but for 9 rows
// and more of many short sequences (64 of 40 with 2 heads: 14.4 / 13.0).  It is causal; of one token that is no matter.
bool kv_chunk_few_rows(const LaunchCtx& c, const KvChunkArgs& a) {
  const long long rows = (long long)a.max_q * a.group;
  if (!(a.causal || a.max_q == 1) || rows > 32) return false;
  return rows <= 8 || !(whole_units(c, a) && 2 * most_units(a) >= c.num_sms);
}

cudaError_t launch_kv_chunk(const LaunchCtx& c, const KvChunkArgs& a, void* ws, int* launches) {
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  if (a.dim == 128) return e5 ? run<128, true>(c, a, ws, launches) : run<128, false>(c, a, ws, launches);
  return e5 ? run<64, true>(c, a, ws, launches) : run<64, false>(c, a, ws, launches);
}

}  // namespace fp8gemm
