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
// Two launches: the up kernel (gate and up products, SwiGLU and quantisation) and
// the down kernel (down product and weighted sum).  For a few tokens each of
// their CTAs routes for itself and the last CTA of an output tile adds what several
// share; for more, two small launches do that.
//
// Bound by the chosen experts' weights, read once, up to some 8 tokens an expert; by
// the conversions and matrix instructions from there on (64 tokens through all 8 of 8 experts:
// 45 GFLOP in 209 us, 0.2 PFLOP/s, where the weights would take 52).  In both product kernels
// the K blocks of all output tiles of all chosen experts form one sequence
// that the CTAs share evenly, in runs, so every SM streams the same number of
// bytes whatever the number of experts.  A warp owns a share of a tile's rows
// and works on its own: one lane asks for the weights ahead (TMA into the
// warp's ring, across tile ends), and the 128-byte swizzle gives every lane its
// share of an m16n8k16 fragment (FP8 codes are exact in FP16) without a bank conflict.  Weight rows are the
// 16-row side, tokens the 8-column side; a contraction's order is free, so a
// lane's share of a row's K block is 32 neighbouring bytes.  A tile that lies in
// several runs is joined from FP32 partials, in CTA order, by the CTA that
// finishes last: results do not depend on timing.
//
// Measured, H 7168, I 2048, 4 of 32 experts: one token (176 MB) 39.5 us, 4.5 TB/s, of
// which the two kernels' starts and joins take 12; 64 tokens (1.41 GB) 237 us, 5.9 TB/s.
#include <type_traits>

#include "common.cuh"
#include "f8_convert.cuh"
#include "moe_few.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// CTAs an SM holds: by registers (and, with 4 fragments of tokens, the down
// kernel's sums).
template <int NT>
constexpr int kPerSm = NT == 4 ? 2 : 3;
constexpr int kMaxPerSm = 3;
constexpr int kMinUnits = 2;  // K blocks a CTA takes at least

// A lane's share of one row's K block, bytes 32 t .. + 31.
struct Chunk {
  uint32_t w[8];
};

// Of an activation row; p: the lane's place in it, in[i]: its i-th 16 bytes are
// inside the row.
__device__ __forceinline__ Chunk load_chunk(const uint8_t* p, const bool (&in)[2]) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in[i]) v = *reinterpret_cast<const uint4*>(p + 16 * i);
    c.w[4 * i] = v.x;
    c.w[4 * i + 1] = v.y;
    c.w[4 * i + 2] = v.z;
    c.w[4 * i + 3] = v.w;
  }
  return c;
}

// Of row r of a weight tile in shared memory, as the TMA swizzles it.
__device__ __forceinline__ Chunk tile_chunk(const uint8_t* tile, int r, int t) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + r * kBlockK + ((2 * t + i) ^ (r & 7)) * 16);
    c.w[4 * i] = v.x;
    c.w[4 * i + 1] = v.y;
    c.w[4 * i + 2] = v.z;
    c.w[4 * i + 3] = v.w;
  }
  return c;
}

// The FP16 pairs of a chunk: word j of it is what a lane holds of k16 step j.
// (The m16n8k32 product of e4m3 operands takes more instructions on this GPU: it
// converts both operands anew for every fragment of tokens.)
struct Halves {
  uint32_t lo[8], hi[8];
};
__device__ __forceinline__ Halves halves(const Chunk& c) {
  Halves h;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h.lo[j] = f8x2_to_f16x2<false>(uint16_t(c.w[j]));
    h.hi[j] = f8x2_to_f16x2<false>(uint16_t(c.w[j] >> 16));
  }
  return h;
}

// One K block of 16 weight rows (lo: rows 0-7, hi: rows 8-15) times up to 8 NT
// tokens: d[n] for the fragments that hold any of the cnt tokens.
template <int NT>
__device__ __forceinline__ void mma_block(float (&d)[NT][4], const Chunk& lo, const Chunk& hi,
                                          const Halves (&x)[NT], int cnt) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) d[n][c] = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a[4] = {
        f8x2_to_f16x2<false>(uint16_t(lo.w[j])), f8x2_to_f16x2<false>(uint16_t(hi.w[j])),
        f8x2_to_f16x2<false>(uint16_t(lo.w[j] >> 16)), f8x2_to_f16x2<false>(uint16_t(hi.w[j] >> 16))};
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n == 0 || 8 * n < cnt) mma_f16(d[n], a, x[n].lo[j], x[n].hi[j]);
  }
}

// ------------------------------------------------------------------ routing
// Pair p = token * k + choice.  A pass is some (at most 8 NT) of the pairs that
// chose one expert, together: expert, first place in the list, pairs.
__device__ __forceinline__ uint32_t pack_pass(int e, int first, int cnt) {
  return uint32_t(e) << 20 | uint32_t(first) << 8 | uint32_t(cnt);
}
struct Pass {
  int e, first, cnt;
  Pass() = default;
  __device__ explicit Pass(uint32_t p) : e(p >> 20), first(p >> 8 & 0xfff), cnt(p & 0xff) {}
};

// Where routing leaves what the product kernels need.
struct Route {
  float* weight;   // [T k]
  int* list;       // [T k] pairs by expert, ascending within each
  uint32_t* pass;  // [T k]
  int* passes;     // how many
};

// Up to kOwnTokens tokens the product kernels route for themselves, each CTA
// into its own shared memory: for one token that takes 1 us of latency where a
// launch before them takes 4.  The work grows with the tokens that a warp has; past
// 8 (two each) a launch of 32 warps is faster.
constexpr int kOwnTokens = 8;
constexpr int kOwnPairs = kOwnTokens * kMoeMaxTopK;

// Scratch of the routing: 4 bytes a pair, 2 an expert, 1 an expert and warp.
__host__ __device__ constexpr int route_scratch(int warps) {
  return 32 * warps * 4 + kMoeMaxExperts * (2 + warps) + 2 * 32 * 4;
}

// A float as an unsigned number of the same order; NaN as -infinity.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (isnan(v)) v = -INFINITY;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);  // -0 and 0 tie
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One warp chooses the experts of token t; kPer values a lane.  ids and w: of
// the token, at lane j its j-th choice.
template <int kPer>
__device__ __forceinline__ void route_token(const float* logits, int E, int k, int renormalise,
                                            int* id, float* w) {
  const int lane = threadIdx.x % 32;
  float v[kPer];
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = lane + 32 * i < E ? logits[lane + 32 * i] : -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < E ? order_key(v[i]) : 0u;  // 0: not to be had
  float first = 0.f, sum = 0.f, mine = 0.f;
  int mine_id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int at = lane;
    float x = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
        x = v[i];
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int win = __reduce_min_sync(0xffffffffu, best == top ? uint32_t(at) : 0xffffffffu);
    x = __shfl_sync(0xffffffffu, x, win % 32);
    if (isnan(x)) x = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (win == lane + 32 * i) key[i] = 0u;
    if (j == 0) first = x;
    const float p = x == -INFINITY ? 0.f : expf(x - first);
    sum += p;
    if (j == lane) {
      mine = p;
      mine_id = win;
    }
  }
  if (!renormalise) {  // over all experts
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += isnan(v[i]) || v[i] == -INFINITY ? 0.f : expf(v[i] - first);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  *id = mine_id;
  *w = sum > 0.f ? __fdiv_rn(mine, sum) : 0.f;
}

// One copy of it for all callers: code that runs once in a launch is fetched line
// by line, and the product kernels wait for it (one token: 42.6 us a call with every
// width inlined at both calls, 40.0 with one function).
__device__ __noinline__ void route_any(const float* logits, int E, int k, int renormalise, int* id,
                                       float* w) {
  if (E <= 32)
    route_token<1>(logits, E, k, renormalise, id, w);
  else if (E <= 128)
    route_token<4>(logits, E, k, renormalise, id, w);
  else
    route_token<kMoeMaxExperts / 32>(logits, E, k, renormalise, id, w);
}

// The whole CTA (kW warps, T k <= 32 kW) routes all tokens; ids_out and w_out
// (the call's outputs) may be null.  Ends with the results written and a barrier.
template <int kW>
__device__ __forceinline__ void route_all(const float* logits, const Route& r, uint8_t* scratch,
                                          int32_t* ids_out, float* w_out, int T, int E, int k,
                                          int renormalise, int per_pass) {
  int* ids = reinterpret_cast<int*>(scratch);                      // [32 kW]
  uint32_t* warp_sum = reinterpret_cast<uint32_t*>(ids + 32 * kW);  // [32]
  uint16_t* first = reinterpret_cast<uint16_t*>(warp_sum + 64);     // [E]
  uint8_t* hist = reinterpret_cast<uint8_t*>(first + kMoeMaxExperts);  // [kW][kMoeMaxExperts]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, P = T * k;
  if (T == 1) {  // every chosen expert has one pair: their order is all there is to find
    if (warp == 0) {
      int id;
      float w;
      route_any(logits, E, k, renormalise, &id, &w);
      int place = 0;
      for (int i = 0; i < k; ++i) place += __shfl_sync(0xffffffffu, id, i) < id;
      if (lane < k) {
        r.list[place] = lane;
        r.pass[place] = pack_pass(id, place, 1);
        r.weight[lane] = w;
        if (ids_out) ids_out[lane] = id;
        if (w_out) w_out[lane] = w;
      }
      if (lane == 0) *r.passes = k;
    }
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < kW * kMoeMaxExperts / 4; i += 32 * kW) reinterpret_cast<uint32_t*>(hist)[i] = 0u;
  for (int t = warp; t < T; t += kW) {
    int id;
    float w;
    route_any(logits + size_t(t) * E, E, k, renormalise, &id, &w);
    if (lane < k) {
      const int p = t * k + lane;
      ids[p] = id;
      r.weight[p] = w;
      if (ids_out) ids_out[p] = id;
      if (w_out) w_out[p] = w;
    }
  }
  __syncthreads();
  // a pair's place: its expert's first, those of the warps before it, those of the lanes before it
  const int p = threadIdx.x, id = p < P ? ids[p] : -1;
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  const int rank = __popc(same & ((1u << lane) - 1u));
  if (id >= 0 && rank == 0) hist[warp * kMoeMaxExperts + id] = uint8_t(__popc(same));
  __syncthreads();
  const int per = ceil_div(E, 32 * kW), e0 = threadIdx.x * per;
  uint32_t sum = 0;  // pairs << 16 | passes of this thread's experts
  for (int e = e0; e < min(E, e0 + per); ++e) {
    int n = 0;
    for (int w = 0; w * 32 < P; ++w) {
      const int h = hist[w * kMoeMaxExperts + e];
      hist[w * kMoeMaxExperts + e] = uint8_t(n);
      n += h;
    }
    first[e] = uint16_t(n);
    sum += uint32_t(n) << 16 | uint32_t(ceil_div(n, per_pass));
  }
  uint32_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += warp_sum[w];
  if (threadIdx.x == 32 * kW - 1) *r.passes = int(upto & 0xffffu);
  uint32_t at = upto - sum;
  for (int e = e0; e < min(E, e0 + per); ++e) {
    const int n = first[e], begin = int(at >> 16), passes = ceil_div(n, per_pass);
    for (int i = 0; i < passes; ++i)
      r.pass[(at & 0xffffu) + i] = pack_pass(e, begin + i * per_pass, min(per_pass, n - i * per_pass));
    first[e] = uint16_t(begin);
    at += uint32_t(n) << 16 | uint32_t(passes);
  }
  __syncthreads();
  if (id >= 0) r.list[first[id] + hist[warp * kMoeMaxExperts + id] + rank] = p;
  __syncthreads();
}

__global__ void __launch_bounds__(1024) moe_route_kernel(const float* __restrict__ logits, Route r,
                                                         int32_t* ids_out, float* w_out, int T,
                                                         int E, int k, int renormalise,
                                                         int per_pass) {
  __shared__ __align__(16) uint8_t scratch[route_scratch(32)];
  griddep_launch_dependents();
  griddep_wait();
  route_all<32>(logits, r, scratch, ids_out, w_out, T, E, k, renormalise, per_pass);
}

// A CTA's own routing.
struct OwnRoute {
  float weight[kOwnPairs];
  int list[kOwnPairs];
  uint32_t pass[kOwnPairs];
  int passes;
  __device__ Route route() { return Route{weight, list, pass, &passes}; }
};
static_assert(kOwnPairs <= 32 * kWarps, "a thread for each pair");
template <int NT>
constexpr bool kOwnRoute = 8 * NT <= kOwnTokens;

// The routing of a launch before, copied into shared memory at `to` (12 bytes a
// pair; 8 without the weights): a change of pass then waits for nothing.
__device__ __forceinline__ Route copy_route(const Route& g, uint8_t* to, int pairs, bool weights) {
  Route r;
  r.pass = reinterpret_cast<uint32_t*>(to);
  r.list = reinterpret_cast<int*>(r.pass + pairs);
  r.weight = reinterpret_cast<float*>(r.list + pairs);
  r.passes = g.passes;
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    r.pass[i] = __ldcg(g.pass + i);  // past the last pass: not used
    r.list[i] = __ldcg(g.list + i);
    if (weights) r.weight[i] = __ldcg(g.weight + i);
  }
  __syncthreads();
  return r;
}

// ------------------------------------------------------------ product kernels
// A CTA's run of the unit sequence, tiles of `len` units each (under 2^31 units: the
// host checks).  Runs are of equal length across tile ends, but where equal parts of
// a tile are at most a unit longer they are taken instead: a run then has one tile
// to join and not two, and a tile fewer runs (5 tokens, H 1040, I 400, 2 of 9
// experts, parts of 3 units for runs of 2: a call takes 15.1 us on the device for 16.6).
struct Run {
  int len, per, parts, u0, u1;  // parts: of a tile; 0: runs of per units
  __device__ Run(int tiles, int len, int ctas, int cta) : len(len) {
    const int units = tiles * len;
    per = max(kMinUnits, int((units + unsigned(ctas) - 1) / unsigned(ctas)));
    parts = len / per;
    if (parts > 0 && ceil_div(len, parts) > per + 1) parts = 0;
    if (parts > 0) {  // tiles * parts <= ctas, since per * ctas >= units
      const int tile = cta / parts, p = cta - tile * parts, least = len / parts, more = len - least * parts;
      u0 = tile < tiles ? tile * len + p * least + min(p, more) : units;
      u1 = tile < tiles ? u0 + least + (p < more) : units;
    } else {
      u0 = int(min((long long)units, (long long)cta * per));
      u1 = int(min((long long)units, (long long)u0 + per));
    }
  }
  __device__ int units() const { return u1 - u0; }
  // The first and the last CTA that a tile lies with.
  __device__ int first(int tile) const { return parts > 0 ? tile * parts : tile * len / per; }
  __device__ int last(int tile) const {
    return parts > 0 ? tile * parts + parts - 1 : (tile * len + len - 1) / per;
  }
};

// One warp's ring of weight tiles.
template <int kStages, int kStageBytes>
struct Ring {
  uint8_t* buf;
  uint64_t* bar;
  uint32_t phases = 0, in_flight = 0;  // bit s: parity to wait for; asked for

  __device__ uint8_t* stage(int s) const { return buf + s * kStageBytes; }
  // Waits for stage s; false, for the whole warp, if that ran out for any of its
  // lanes (or another warp's wait did).
  __device__ bool wait(int s, int* gave_up, int* status, unsigned long long limit_ns) {
    if (!__all_sync(0xffffffffu, mbar_wait_within(&bar[s], phases >> s & 1, gave_up, limit_ns))) {
      // results are void; what is still in flight lands before the CTA ends
      *reinterpret_cast<volatile int*>(gave_up) = 1;
      raise_status(status, FP8GEMM_ERR_TIMEOUT);
      for (int k = 0; k < kStages; ++k)
        if (in_flight >> k & 1) mbar_drain(&bar[k], phases >> k & 1);
      return false;
    }
    phases ^= 1u << s;
    in_flight &= ~(1u << s);
    return true;
  }
};

struct Shared {
  uint64_t bars[kWarps][4];
  int gave_up, last_one;  // a wait ran out; this CTA joins
};

__device__ __forceinline__ uint8_t* init_shared(Shared& sh, uint8_t* raw, const CUtensorMap* map) {
  if (threadIdx.x == 0) {
    sh.gave_up = 0;
    for (int i = 0; i < kWarps * 4; ++i) mbar_init(&sh.bars[0][i], 1);
    fence_mbar_init();
    tma_prefetch_desc(map);
  }
  __syncthreads();
  return raw + (1024u - (smem_addr(raw) & 1023u)) % 1024u;
}

// Four columns of the partials of CTAs first .. last, added in that order, eight
// of their loads in flight.
__device__ __forceinline__ float4 sum_partials(const float* parts, size_t size, int first, int last) {
  constexpr int kAtOnce = 8;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q0 = first; q0 <= last; q0 += kAtOnce) {
    float4 v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int q = q0 + i;
      v[i] = q <= last ? __ldcg(reinterpret_cast<const float4*>(
                             parts + size_t(2 * q + (q == first ? 1 : 0)) * size))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      sum.x += v[i].x;
      sum.y += v[i].y;
      sum.z += v[i].z;
      sum.w += v[i].w;
    }
  }
  return sum;
}

__device__ __forceinline__ void store_bf16x4(__nv_bfloat16* to, const float4& v) {
  *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2_bits(v.x, v.y), bf16x2_bits(v.z, v.w));
}

// x / (1 + e^-x), to some 2^-21 of it (h is rounded to 4 bits next).  This and the
// quantisation run once in a CTA, right behind its last copy, from instructions that
// are not in any cache yet: the division's and the exponential's full sequences
// in their place cost a call 2 us.
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// Gate and up products.  Unit: one K block of a tile (pass, 128 hidden
// columns); warp w takes hidden columns 32 w .. + 31 of it, rows of gate and of
// up alike, so that SwiGLU stays within a lane.
//   partial: [warp][fragment 0-3][n][element][lane] floats
template <int NT>
constexpr int kUpStages = NT == 4 ? 3 : 2;

template <int NT>
__global__ void __launch_bounds__(kThreads, kPerSm<NT>) moe_up_kernel(const MoeArgs a, const Route given,
                                                             const __grid_constant__ CUtensorMap map,
                                                             uint8_t* __restrict__ H8,
                                                             float* __restrict__ sH, int* counters,
                                                             float* parts, int* status) {
  constexpr int kPart = kWarps * 4 * NT * 4 * 32;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  __shared__ std::conditional_t<kOwnRoute<NT>, OwnRoute, int> mine;
  __shared__ float amaxes[kWarps][8 * NT];
  __shared__ __align__(16) uint8_t codes[8 * NT][kBlockK];
  uint8_t* rings = init_shared(sh, raw, &map);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int Kb = ceil_div(a.H, kBlockK), Ib = ceil_div(a.I, kBlockK), Rb = ceil_div(2 * a.I, kBlockK);
  Ring<kUpStages<NT>, 64 * kBlockK> ring{rings + warp * kUpStages<NT> * 64 * kBlockK, sh.bars[warp]};
  griddep_wait();
  griddep_launch_dependents();  // all before this kernel is complete: the next may read weights
  Route r = given;
  if constexpr (kOwnRoute<NT>) {  // into the rings' memory first: nothing has been asked for yet
    r = mine.route();
    const bool out = blockIdx.x == 0;
    route_all<kWarps>(a.logits, r, rings, out ? a.ids : nullptr, out ? a.weights : nullptr, a.T, a.E,
                      a.k, a.renormalise, 8 * NT);
    fence_proxy_async_smem();
    __syncthreads();
  } else {
    r = copy_route(given, rings + kWarps * kUpStages<NT> * 64 * kBlockK, a.T * a.k, false);
  }
  const Run run(*r.passes * Ib, Kb, gridDim.x, blockIdx.x);
  int left = run.units();
  if (left == 0) return;

  // the tile and K block in use, and those asked for (kUpStages ahead)
  int tile = run.u0 / Kb, kb = run.u0 - tile * Kb;
  int pi = tile / Ib, ib = tile - pi * Ib;
  int ask_left = left, ask_pi = pi, ask_ib = ib, ask_kb = kb, ask_stage = 0;
  int ask_row = Pass(r.pass[pi]).e * 2 * a.I + ib * kBlockK + 32 * warp;
  auto fetch = [&]() {
    if (ask_left == 0) return;
    --ask_left;
    ring.in_flight |= 1u << ask_stage;
    if (lane == 0) {
      uint8_t* s = ring.stage(ask_stage);
      mbar_arrive_expect_tx(&ring.bar[ask_stage], 64 * kBlockK);
      tma_load_2d(s, &map, &ring.bar[ask_stage], ask_kb * kBlockK, ask_row);
      tma_load_2d(s + 32 * kBlockK, &map, &ring.bar[ask_stage], ask_kb * kBlockK, ask_row + a.I);
    }
    ask_stage = ask_stage + 1 == kUpStages<NT> ? 0 : ask_stage + 1;
    if (++ask_kb == Kb && ask_left > 0) {
      ask_kb = 0;
      if (++ask_ib == Ib) {
        ask_ib = 0;
        ++ask_pi;
      }
      ask_row = Pass(r.pass[ask_pi]).e * 2 * a.I + ask_ib * kBlockK + 32 * warp;
    }
  };
#pragma unroll
  for (int i = 0; i < kUpStages<NT>; ++i) fetch();

  // What a unit needs besides weights.  Columns without a pair take the
  // pass's last one: their results are not used.
  Pass at;
  const uint8_t* x[NT];
  const float* sx[NT][2];
  const float *sg, *su[2];
  auto enter_pass = [&]() {
    at = Pass(r.pass[pi]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x[n] = a.A + size_t(r.list[at.first + min(8 * n + g, at.cnt - 1)] / a.k) * a.H + 32 * t;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        sx[n][c] = a.sA + size_t(r.list[at.first + min(8 * n + 2 * t + c, at.cnt - 1)] / a.k) * Kb;
    }
  };
  auto enter_tile = [&]() {
    const float* s = a.s1 + size_t(at.e) * Rb * Kb;
    sg = s + size_t(ib) * Kb;
#pragma unroll
    for (int m = 0; m < 2; ++m)
      su[m] = s + size_t(min((a.I + ib * kBlockK + 32 * warp + 16 * m) / kBlockK, Rb - 1)) * Kb;
  };
  // loaded a unit ahead of its use
  Halves xc[NT];
  Chunk next_x[NT];
  float sxk[NT][2], next_sx[NT][2], sw[3], next_sw[3];
  auto load_side = [&](int k) {
    const bool in[2] = {k * kBlockK + 32 * t < a.H, k * kBlockK + 32 * t + 16 < a.H};
    next_sw[0] = sg[k];
    next_sw[1] = su[0][k];
    next_sw[2] = su[1][k];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= at.cnt) break;
      next_x[n] = load_chunk(x[n] + k * kBlockK, in);
      next_sx[n][0] = sx[n][0][k];
      next_sx[n][1] = sx[n][1][k];
    }
  };
  enter_pass();
  enter_tile();
  load_side(kb);

  float acc[4][NT][4] = {};
  int stage = 0;
  bool dead = false;
  while (true) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xc[n] = halves(next_x[n]);
      sxk[n][0] = next_sx[n][0];
      sxk[n][1] = next_sx[n][1];
    }
#pragma unroll
    for (int m = 0; m < 3; ++m) sw[m] = next_sw[m];
    if (kb + 1 < Kb && left > 1) load_side(kb + 1);
    // After a wait that ran out the warp only keeps the others' barriers company.
    dead = dead || !ring.wait(stage, &sh.gave_up, status, a.wait_ns);
    const uint8_t* w = ring.stage(stage);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const Chunk lo = tile_chunk(w, 16 * m + g, t), hi = tile_chunk(w, 16 * m + 8 + g, t);
      float d[NT][4];
      mma_block<NT>(d, lo, hi, xc, at.cnt);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[m][n][c] = fmaf(d[n][c], sxk[n][c & 1] * sw[m < 2 ? 0 : m - 1], acc[m][n][c]);
      }
    }
    __syncwarp();  // the stage has been read
    if (!dead) fetch();
    stage = stage + 1 == kUpStages<NT> ? 0 : stage + 1;
    ++kb;
    --left;
    if (kb < Kb && left > 0) continue;

    const int tile0 = tile * Kb;
    // the run's share of this tile is done
    const bool whole = tile0 >= run.u0 && tile0 + Kb <= run.u1;
    const int first = run.first(tile), last = run.last(tile);
    if (!whole) {
      float* part = parts + size_t(2 * blockIdx.x + (tile0 >= run.u0 ? 1 : 0)) * kPart +
                    warp * (4 * NT * 4 * 32) + lane;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) part[((m * NT + n) * 4 + c) * 32] = acc[m][n][c];
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        sh.last_one = atomic_add_acq_rel_gpu(counters + first, 1) == last - first;
        if (sh.last_one) counters[first] = 0;
      }
      __syncthreads();
      if (sh.last_one) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (8 * n >= at.cnt) break;
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.f;
#pragma unroll 4
          for (int q = first; q <= last; ++q) {
            const float* p = parts + size_t(2 * q + (q == first ? 1 : 0)) * kPart +
                             warp * (4 * NT * 4 * 32) + lane;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int c = 0; c < 4; ++c) acc[m][n][c] += __ldcg(p + ((m * NT + n) * 4 + c) * 32);
          }
        }
      }
    }
    if (whole || sh.last_one) {  // SwiGLU and the 1x128 quantisation of the tile
      const int i0 = ib * kBlockK;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float gate = acc[m][n][c];
            float h = silu(gate) * acc[2 + m][n][c];
            if (i0 + 32 * warp + 16 * m + g + 8 * (c >> 1) >= a.I) h = 0.f;
            acc[m][n][c] = h;
            top[c & 1] = fmaxf(top[c & 1], fabsf(h));
          }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], o));
          if (g == 0) amaxes[warp][8 * n + 2 * t + c] = top[c];
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int j = 8 * n + 2 * t + c;
          float top = 0.f;
#pragma unroll
          for (int w2 = 0; w2 < kWarps; ++w2) top = fmaxf(top, amaxes[w2][j]);
          const float s = __fdiv_rn(top, kE4M3Max);
          if (j < at.cnt && warp == 0 && g == 0)
            sH[size_t(r.list[at.first + j]) * Ib + ib] = s;
          // h / s without the division's sequence (see silu): both times a power of two that
          // brings s into the range of the corrected quotient (h that this makes too small
          // to hold has the code 0, and so has a block whose s itself is: h pre < 2^-40)
          const float pre = s < 1e-25f ? 0x1p100f : s > 1e25f ? 0x1p-100f : 1.f;
          const Reciprocal d = reciprocal(s != 0.f ? s * pre : 1.f);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              codes[j][32 * warp + 16 * m + 8 * e + g] =
                  uint8_t(cvt_f8x2<false>(quotient(acc[m][n][2 * e + c] * pre, d), 0.f));
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < at.cnt * (kBlockK / 16); i += kThreads) {
        const int j = i / (kBlockK / 16), c = i % (kBlockK / 16) * 16;
        if (i0 + c < a.I)
          *reinterpret_cast<uint4*>(H8 + size_t(r.list[at.first + j]) * a.I + i0 + c) =
              *reinterpret_cast<const uint4*>(&codes[j][c]);
      }
      __syncthreads();  // amaxes and codes are free
    }
    if (left == 0) break;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.f;
    kb = 0;
    ++tile;
    if (++ib == Ib) {
      ib = 0;
      ++pi;
      enter_pass();
    }
    enter_tile();
    load_side(0);
  }
}

// The down kernel's partials hold 128 bytes a token and warp.  For a few tokens the
// last CTA of a tile adds them; for more that took one CTA 20 us at the end of a
// call (64 tokens, 9 partials of 32 KB), so a launch of many CTAs does it.
template <int NT>
constexpr bool kJoinHere = NT == 1;

// Stages of a warp's ring of 4 KB tiles: beside the tokens' sums two leave room for
// three CTAs (16 tokens through 4 of 32 experts, H 7168, I 2048: a call takes 223 us
// with two, 231 with four).
template <int NT>
constexpr int kDownStages = NT == 2 ? 2 : 4;

// Down product and weighted sum.  Unit: one K block of one pass for a tile of
// 128 output columns; warp w takes columns 32 w .. + 31 and keeps a sum per token
// in shared memory that no other warp touches.
//   partial: [warp][token][32] floats
constexpr int kSumRow = 36;  // floats from token to token: lanes of a fragment hit all banks

template <int NT>
__global__ void __launch_bounds__(kThreads, kPerSm<NT>) moe_down_kernel(const MoeArgs a, const Route given,
                                                               const __grid_constant__ CUtensorMap map,
                                                               const uint8_t* H8, const float* sH,
                                                               int* counters, float* parts,
                                                               int* status) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  __shared__ std::conditional_t<kOwnRoute<NT>, OwnRoute, int> mine;
  uint8_t* rings = init_shared(sh, raw, &map);
  float* all_sums = reinterpret_cast<float*>(rings + kWarps * kDownStages<NT> * 32 * kBlockK);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int Kb = ceil_div(a.I, kBlockK), Hb = ceil_div(a.H, kBlockK);
  float* sums = all_sums + warp * a.T * kSumRow;
  for (int i = lane; i < a.T * kSumRow; i += 32) sums[i] = 0.f;
  Ring<kDownStages<NT>, 32 * kBlockK> ring{rings + warp * kDownStages<NT> * 32 * kBlockK, sh.bars[warp]};
  // The up kernel let this one start after everything before it was complete:
  // logits, routing and weights may be read, the hidden activations not yet.
  Route r = given;
  if constexpr (kOwnRoute<NT>) {
    r = mine.route();
    route_all<kWarps>(a.logits, r, rings, nullptr, nullptr, a.T, a.E, a.k, a.renormalise, 8 * NT);
    fence_proxy_async_smem();
    __syncthreads();
  } else {
    r = copy_route(given, reinterpret_cast<uint8_t*>(all_sums + kWarps * a.T * kSumRow), a.T * a.k, true);
  }
  const int passes = *r.passes;
  const int per_tile = passes * Kb;
  const Run run(Hb, per_tile, gridDim.x, blockIdx.x);
  int left = run.units();
  if (left == 0) {
    griddep_wait();
    return;
  }
  int tile = run.u0 / per_tile, pi = (run.u0 - tile * per_tile) / Kb, kb = run.u0 % Kb;
  int ask_left = left, ask_tile = tile, ask_pi = pi, ask_kb = kb, ask_stage = 0;
  int ask_row = Pass(r.pass[pi]).e * a.H + tile * kBlockK + 32 * warp;
  auto fetch = [&]() {
    if (ask_left == 0) return;
    --ask_left;
    ring.in_flight |= 1u << ask_stage;
    if (lane == 0) {
      mbar_arrive_expect_tx(&ring.bar[ask_stage], 32 * kBlockK);
      tma_load_2d(ring.stage(ask_stage), &map, &ring.bar[ask_stage], ask_kb * kBlockK, ask_row);
    }
    ask_stage = (ask_stage + 1) % kDownStages<NT>;
    if (++ask_kb == Kb && ask_left > 0) {
      ask_kb = 0;
      if (++ask_pi == passes) {
        ask_pi = 0;
        ++ask_tile;
      }
      ask_row = Pass(r.pass[ask_pi]).e * a.H + ask_tile * kBlockK + 32 * warp;
    }
  };
#pragma unroll
  for (int i = 0; i < kDownStages<NT>; ++i) fetch();
  // With the sum in a launch of its own, that may come early.  The next call's
  // routing may not: it takes a whole SM's registers, which this kernel's CTAs would
  // go without (64 tokens: that cost a call 39 us).
  if constexpr (!kJoinHere<NT>) griddep_launch_dependents();
  griddep_wait();

  // What a unit needs besides weights.  Columns without a pair take the
  // pass's last one: their results are not used.
  Pass at;
  const uint8_t* x[NT];
  const float* sx[NT][2];
  const float* sw;
  auto enter = [&]() {
    at = Pass(r.pass[pi]);
    sw = a.s2 + (size_t(at.e) * Hb + tile) * Kb;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x[n] = H8 + size_t(r.list[at.first + min(8 * n + g, at.cnt - 1)]) * a.I + 32 * t;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        sx[n][c] = sH + size_t(r.list[at.first + min(8 * n + 2 * t + c, at.cnt - 1)]) * Kb;
    }
  };
  // loaded a unit ahead of its use
  Halves xc[NT];
  Chunk next_x[NT];
  float sxk[NT][2], next_sx[NT][2], next_sw = 0.f;
  auto load_side = [&](int k) {
    const bool in[2] = {k * kBlockK + 32 * t < a.I, k * kBlockK + 32 * t + 16 < a.I};
    next_sw = sw[k];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= at.cnt) break;
      next_x[n] = load_chunk(x[n] + k * kBlockK, in);
      next_sx[n][0] = sx[n][0][k];
      next_sx[n][1] = sx[n][1][k];
    }
  };
  enter();
  load_side(kb);

  float acc[2][NT][4] = {};
  int stage = 0;
  bool dead = false;
  while (true) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xc[n] = halves(next_x[n]);
      sxk[n][0] = next_sx[n][0] * next_sw;
      sxk[n][1] = next_sx[n][1] * next_sw;
    }
    if (kb + 1 < Kb && left > 1) load_side(kb + 1);
    dead = dead || !ring.wait(stage, &sh.gave_up, status, a.wait_ns);
    const uint8_t* w = ring.stage(stage);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const Chunk lo = tile_chunk(w, 16 * m + g, t), hi = tile_chunk(w, 16 * m + 8 + g, t);
      float d[NT][4];
      mma_block<NT>(d, lo, hi, xc, at.cnt);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = fmaf(d[n][c], sxk[n][c & 1], acc[m][n][c]);
      }
    }
    __syncwarp();  // the stage has been read
    if (!dead) fetch();
    stage = (stage + 1) % kDownStages<NT>;
    ++kb;
    --left;
    if (kb < Kb && left > 0) continue;
    const int this_tile = tile;
    const Pass done = at;
    kb = 0;
    if (++pi == passes) {
      pi = 0;
      ++tile;
    }
    if (left > 0) {  // the next pass's activations are on their way meanwhile
      enter();
      load_side(0);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= done.cnt) break;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = 8 * n + 2 * t + c;
        if (j < done.cnt) {
          const int pair = r.list[done.first + j];
          const float wt = r.weight[pair];
          float* s = sums + pair / a.k * kSumRow + g;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[16 * m + 8 * e] = fmaf(acc[m][n][2 * e + c], wt, s[16 * m + 8 * e]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) acc[m][n][c] = acc[m][n][2 + c] = 0.f;
      }
    }
    __syncwarp();
    if (left > 0 && tile == this_tile) continue;

    const int tile0 = this_tile * per_tile;
    // the run's share of this tile is done
    const bool whole = tile0 >= run.u0 && tile0 + per_tile <= run.u1;
    const int first = run.first(this_tile), last = run.last(this_tile);
    const size_t part_size = size_t(kWarps) * a.T * 32;
    const int h0 = this_tile * kBlockK + 32 * warp;
    if (!whole) {
      float* part = parts + (2 * blockIdx.x + (tile0 >= run.u0 ? 1 : 0)) * part_size + warp * a.T * 32;
      for (int i = lane; i < a.T * 8; i += 32)
        reinterpret_cast<float4*>(part)[i] =
            *reinterpret_cast<const float4*>(sums + i / 8 * kSumRow + i % 8 * 4);
      if constexpr (kJoinHere<NT>) {
        __syncthreads();
        if (threadIdx.x == 0) {
          sh.last_one = atomic_add_acq_rel_gpu(counters + first, 1) == last - first;
          if (sh.last_one) counters[first] = 0;
        }
        __syncthreads();
        if (sh.last_one)
          for (int i = lane; i < a.T * 8; i += 32) {
            const float4 v = sum_partials(parts + warp * a.T * 32 + 4 * i, part_size, first, last);
            *reinterpret_cast<float4*>(sums + i / 8 * kSumRow + i % 8 * 4) = v;
          }
        __syncwarp();
      }
    }
    if (whole || (kJoinHere<NT> && sh.last_one))
      for (int i = lane; i < a.T * 8; i += 32) {
        const int h = h0 + i % 8 * 4;
        if (h >= a.H) continue;  // H is a multiple of 16
        store_bf16x4(a.D + size_t(i / 8) * a.H + h,
                     *reinterpret_cast<const float4*>(sums + i / 8 * kSumRow + i % 8 * 4));
      }
    if (left == 0) break;
    __syncthreads();  // last_one is free
    for (int i = lane; i < a.T * kSumRow; i += 32) sums[i] = 0.f;
    __syncwarp();
  }
}

// The tiles that lie in several runs of the down kernel: the sum of their
// partials in CTA order.  Grid (tiles, tokens / 4); a thread has 4 columns of one token.
__global__ void __launch_bounds__(128) moe_sum_kernel(const MoeArgs a, const int* passes,
                                                      const float* parts, int ctas) {
  const int Kb = ceil_div(a.I, kBlockK), Hb = ceil_div(a.H, kBlockK);
  const int tile = blockIdx.x, token = blockIdx.y * 4 + threadIdx.x / 32;
  const int warp = threadIdx.x % 32 / 8, c = threadIdx.x % 8;  // of the down kernel
  const int per_tile = __ldcg(passes) * Kb;  // routing was complete before the down kernel began
  const Run run(Hb, per_tile, ctas, 0);
  const int first = run.first(tile), last = run.last(tile);
  const int h = tile * kBlockK + 32 * warp + 4 * c;
  griddep_wait();
  if (first == last || token >= a.T || h >= a.H) return;
  store_bf16x4(a.D + size_t(token) * a.H + h,
               sum_partials(parts + (size_t(warp) * a.T + token) * 32 + 4 * c,
                            size_t(kWarps) * a.T * 32, first, last));
}

// ------------------------------------------------------------------- launches
// Fragments of 8 tokens that a pass takes.  Two keep three CTAs on an SM; four
// save passes over the weights where an expert has more than 32 tokens as a rule
// (64 tokens, H 7168, I 2048: through 8 of 32 experts, 16 tokens each, 313 us with
// two, 351 with four; 4 of 8, 32 each, 154 and 161; 8 of 8, 64 each, 239 and 209).
constexpr int kMaxFragments = 4;
int fragments(const MoeArgs& a) {
  return a.T <= 8 ? 1 : a.T * a.k <= 32 * a.E ? 2 : 4;
}

// Shared memory of an SM, and the most a CTA may ask for.
constexpr size_t kSmemPerSm = 228 * 1024, kMaxSmem = 200 * 1024;
// CTAs that an SM holds: a CTA takes 1 KB of the system's beside its own.
int per_sm(int most, size_t dynamic, size_t fixed) {
  return max(1, min(most, int(kSmemPerSm / (dynamic + fixed + 1024))));
}

struct Layout {
  size_t counters, h8, sh, weight, list, pass, passes, up, down, total;
};

// Places for the most tokens and choices: only I changes them, so that a stream's
// buffer stays where it is (a captured graph holds its address).
Layout layout(const LaunchCtx& c, const MoeArgs& a) {
  const size_t P = size_t(kMoeMaxTokens) * kMoeMaxTopK, grid = size_t(kMaxPerSm) * c.num_sms;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  Layout l;
  l.counters = take(2 * grid * 4);  // first: zeros that one call leaves are what the next one finds
  l.h8 = take(P * a.I);
  l.sh = take(P * ceil_div(a.I, kBlockK) * 4);
  l.weight = take(P * 4);
  l.list = take(P * 4);
  l.pass = take(P * 4);
  l.passes = take(4);
  l.up = take(2 * grid * kWarps * 4 * kMaxFragments * 4 * 32 * 4);
  l.down = take(2 * grid * kWarps * kMoeMaxTokens * 32 * 4);
  l.total = at;
  return l;
}

template <int NT>
cudaError_t launch_nt(const LaunchCtx& c, const MoeArgs& a, const Route& r, char* ws,
                      const Layout& l) {
  CUtensorMap m1, m2;
  if (!make_tmap_u8_sw128(&m1, a.W1, uint64_t(a.E) * 2 * a.I, a.H, 32) ||
      !make_tmap_u8_sw128(&m2, a.W2, uint64_t(a.E) * a.H, a.I, 32))
    return cudaErrorInvalidValue;
  uint8_t* H8 = reinterpret_cast<uint8_t*>(ws + l.h8);
  float* sH = reinterpret_cast<float*>(ws + l.sh);
  int* counters = reinterpret_cast<int*>(ws + l.counters);
  const size_t pairs = kOwnRoute<NT> ? 0 : size_t(a.T) * a.k;
  const size_t up_smem = 1024 + size_t(kWarps) * kUpStages<NT> * 64 * kBlockK + 8 * pairs;
  const size_t down_smem = 1024 + size_t(kWarps) * kDownStages<NT> * 32 * kBlockK +
                           size_t(kWarps) * a.T * kSumRow * 4 + 12 * pairs;
  const int up_per_sm = per_sm(kPerSm<NT>, up_smem, 3 * 1024);
  const int down_per_sm = per_sm(kPerSm<NT>, down_smem, 2 * 1024);
  auto up = moe_up_kernel<NT>;
  auto down = moe_down_kernel<NT>;
  static SmemLimit up_limit, down_limit;
  if (cudaError_t e = up_limit.raise(c, reinterpret_cast<const void*>(up), kMaxSmem)) return e;
  if (cudaError_t e = down_limit.raise(c, reinterpret_cast<const void*>(down), kMaxSmem)) return e;
  if constexpr (!kOwnRoute<NT>)
    if (cudaError_t e = launch_dependent(c, moe_route_kernel, 1, 1024, 0, a.logits, r, a.ids,
                                         a.weights, a.T, a.E, a.k, a.renormalise, 8 * NT))
      return e;
  if (cudaError_t e = launch_dependent(c, up, up_per_sm * c.num_sms, kThreads, up_smem, a, r, m1, H8, sH, counters,
                                       reinterpret_cast<float*>(ws + l.up), c.status))
    return e;
  float* parts = reinterpret_cast<float*>(ws + l.down);
  const int ctas = down_per_sm * c.num_sms;
  if (cudaError_t e = launch_dependent(c, down, ctas, kThreads, down_smem, a, r, m2, H8, sH,
                                       counters + kMaxPerSm * c.num_sms, parts, c.status))
    return e;
  if constexpr (kJoinHere<NT>) return cudaSuccess;
  return launch_dependent(c, moe_sum_kernel, dim3(ceil_div(a.H, kBlockK), ceil_div(a.T, 4)), 128, 0, a,
                          r.passes, parts, ctas);
}

}  // namespace

size_t moe_few_workspace_bytes(const LaunchCtx& c, const MoeArgs& a) { return layout(c, a).total; }

cudaError_t launch_moe_few(const LaunchCtx& c, const MoeArgs& a, void* workspace, int* launches) {
  char* ws = static_cast<char*>(workspace);
  const Layout l = layout(c, a);
  const Route r{reinterpret_cast<float*>(ws + l.weight), reinterpret_cast<int*>(ws + l.list),
                reinterpret_cast<uint32_t*>(ws + l.pass), reinterpret_cast<int*>(ws + l.passes)};
  *launches = a.T <= kOwnTokens ? 2 : 4;
  switch (fragments(a)) {
    case 1: return launch_nt<1>(c, a, r, ws, l);
    case 2: return launch_nt<2>(c, a, r, ws, l);
    default: return launch_nt<4>(c, a, r, ws, l);
  }
}

}  // namespace fp8gemm
