// kv_attention.cu -- attention of a sequence's newest tokens over its paged
// FP8 cache (kv_cache.cu has the layout).
//
//   o = sum_j p_j v_j,  p = softmax over the visible j of (scale q . k_j)
//
// The query of new token i of n sees the first len - n + 1 + i cached tokens
// (its own among them); a row that sees none gives zeros.  Query heads h g ..
// h g + g - 1 read the cached head h, so their rows share every byte of it.
//
// Bound by the cache's bytes: each is read once.  A warp works on its own: one
// lane asks for the tiles ahead (TMA into the warp's ring in shared memory, one
// mbarrier a stage), and the 128-byte swizzle lets every lane read its share of
// a tensor-core fragment as 16 neighbouring bytes without a bank conflict.  Both products
// are taken transposed so that tokens (and the head's dimension) fill the
// 16-row side of m16n8k16 and 8 query rows the other:
//   S^T [16 tokens, 8 rows] = K [16, dim] Q^T      O^T [dim, 8 rows] += V^T [dim, 16] P^T
// The order of a contraction is free, so the dimension is dealt to the
// fragment's k index such that a lane's share of a key is 16 neighbouring bytes, and the
// output dimension to V^T's rows such that a lane's share of a value is too.
// FP8 codes are exact in FP16; q is shifted by a power of two per row to use
// FP16's range (BF16 has fewer mantissa bits); p is rounded to FP16 (11 bits where it
// is 2^-25 of the largest or more; the BF16 output has 8).  Scores, statistics, sums and
// the output accumulate in FP32; a tile's scales are applied to its FP32 products, the
// values' as they are added to O: a scale inside p would take p out of FP16's range
// where neighbouring blocks' scales differ (64 ragged sequences with 8 rows a head: 100 us
// either way; 32 rows, which the products bound: 195 with the scale in p, 208 so).
// Measured: 64 ragged sequences of up to 8192 tokens, 8 heads of 128 (584 MB) 100 us, 5.8
// TB/s; one of 131077 with 16 rows a head (268 MB) 55 us, 4.9 TB/s, of which the start
// takes 5 and the join of the CTAs' results 6.  Past 16 rows a head conversions and
// products bind (64 sequences with 32 rows: 208 us).
#include <cfloat>

#include "common.cuh"
#include "f8_convert.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kFrag = 16;          // tokens of a fragment
constexpr int kTok = 2 * kFrag;    // tokens of a tile: two fragments, whose chains of
                                   // dependent instructions run side by side
constexpr int kRows = 8;   // query rows per fragment
// Work is shared out in tiles.  A CTA's least share is 256 tokens: fewer would
// cost more to join than to do.
constexpr int kMinTiles = 8;
// What beginning and joining an item costs, in tiles (about 5 us, in which the
// warps of a CTA would do four each).  It counts in a CTA's share as if the item
// began with that many tiles more: 64 ragged sequences took 120 us with equal
// shares of the tiles alone, for which the CTAs with many short items were late, and
// 100 us with it (16 ragged ones: 35.5 us with 12 for it, 34.6 with 16, 33.9 with 20; the 64:
// 99.7, 100.0, 100.3).
constexpr int kItemCost = 16;
constexpr int kStages = 2;  // tiles of a warp in shared memory
constexpr float kNone = -FLT_MAX;  // the maximum of nothing: not above any score
// p is held times 2^kLift, and the running maximum may lag by 2^kLazy: FP16's largest
// numbers are in use, so that p keeps its 11 bits down to 2^-(14 + kLift) of the largest one
// and is lost below 2^-(25 + kLift) only (131072 tokens there are 2^-19 of the sum).  The lift
// is added to the difference of score and maximum: it would be lost in a large maximum.
constexpr float kLazy = 4.f, kLift = 11.f;
constexpr float kUnlift = 1.f / 2048;  // 2^-kLift

// Transposes an 8x8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^x to FP32's rounding (relative error 2^-22).
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A tile of one head: 32 tokens, 16-byte chunk c of token r at chunk c ^ (r & 7) of
// its 128 bytes (64-byte tokens: c ^ (r / 2 & 3), as the TMA writes them).  With lane
// = 4 g + t, a lane's share of each fragment is
//   keys    tokens g and g + 8, bytes (dim / 4) t .. + dim / 4 - 1
//   values  tokens 2t, 2t + 1, 2t + 8, 2t + 9, bytes (dim / 8) g .. + dim / 8 - 1
template <int kDim>
struct Stage {
  uint8_t k[kTok][kDim];
  uint8_t v[kTok][kDim];
};

// Key chunk c (of dim / 64) of token g + 8 i of fragment h.
template <int kDim>
__device__ __forceinline__ uint4 key_chunk(const Stage<kDim>& s, int h, int i, int c, int g, int t) {
  const int r = kFrag * h + 8 * i + g;
  if constexpr (kDim == 128)
    return *reinterpret_cast<const uint4*>(&s.k[r][((2 * t + c) ^ g) * 16]);
  else
    return *reinterpret_cast<const uint4*>(&s.k[r][(t ^ (g / 2)) * 16]);
}

// The lane's bytes of its p-th value token of fragment h.
template <int kDim>
__device__ __forceinline__ void value_bytes(const Stage<kDim>& s, int h, int p, int g, int t,
                                            uint32_t (&v)[kDim / 32]) {
  const int r = kFrag * h + 2 * t + (p & 1) + 8 * (p >> 1);
  if constexpr (kDim == 128) {
    const uint4 x = *reinterpret_cast<const uint4*>(&s.v[r][(g ^ (2 * t + (p & 1))) * 16]);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(&s.v[r][((g / 2) ^ t) * 16 + g % 2 * 8]);
    v[0] = x.x;
    v[1] = x.y;
  }
}

// The queries of 8 rows as the k16 x n8 fragments that match Tile's keys, and
// what their products have to be multiplied by (rows 2t and 2t + 1 of this lane).
template <int kDim>
struct Queries {
  uint32_t b[kDim / 16][2];
  float mul[2];
};

// A lane's share of one row's query, as it lies; zeros without a row.
template <int kDim>
struct RawQuery {
  Raw8<__nv_bfloat16> r[kDim / 64][2];
};

template <int kDim>
__device__ __forceinline__ RawQuery<kDim> load_query(const __nv_bfloat16* row, int t) {
  RawQuery<kDim> q;
#pragma unroll
  for (int c = 0; c < kDim / 64; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      zero8(q.r[c][e]);
      if (row) q.r[c][e] = load8(row + (kDim / 4) * t + 16 * c + 8 * e);
    }
  return q;
}

template <int kDim>
__device__ __forceinline__ void take_queries(Queries<kDim>& q, const RawQuery<kDim>& raw,
                                             float scale_log2, int t) {
  float x[kDim / 64][16];
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < kDim / 64; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float f[8];
      unpack8(raw.r[c][e], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[c][8 * e + i] = f[i];
        top = fmaxf(top, fabsf(f[i]));
      }
    }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 2^e brings the row's largest value into [2^10, 2^11); rows below 2^-117
  // (zeros among them) take the largest shift that is a normal number
  const int exp = max(int(__float_as_uint(top) >> 23), 10);
  const float up = __uint_as_float(uint32_t(264 - exp) << 23);    // 2^(10 - (exp - 127))
  const float down = __uint_as_float(uint32_t(exp - 10) << 23) ;  // its reciprocal
#pragma unroll
  for (int ks = 0; ks < kDim / 16; ++ks) {
    const float* p = &x[ks / 4][ks % 4 * 4];
    q.b[ks][0] = f16x2_bits(p[0] * up, p[1] * up);
    q.b[ks][1] = f16x2_bits(p[2] * up, p[3] * up);
  }
  const float mul = down * scale_log2;  // held by the lanes of row g: fetch rows 2t and 2t + 1
  q.mul[0] = __shfl_sync(0xffffffffu, mul, 8 * t);
  q.mul[1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
}

// Running softmax of a lane's two rows and its share of O^T: o[j] holds dimensions
// (dim/8) g + 2j (rows 2t, 2t + 1) and + 1 (rows 2t, 2t + 1).
template <int kDim>
struct State {
  float m[2], l[2];  // l: this lane's tokens only, times 2^kLift
  float o[kDim / 16][4];
};

template <int kDim>
__device__ __forceinline__ void clear(State<kDim>& s) {
  s.m[0] = s.m[1] = 0.f;  // the first tile sets it
  s.l[0] = s.l[1] = 0.f;
#pragma unroll
  for (int j = 0; j < kDim / 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s.o[j][e] = 0.f;
}

// A tile that some rows do not see whole may hold values (or have a scale) that are not
// finite, of tokens that some row does not see, and 0 times one is NaN.  Whether it does:
// lane l looks at token l, if that is such a one.
template <int kDim, bool kE5M2>
__device__ __forceinline__ bool any_not_finite(const Stage<kDim>& x, bool mine, int lane,
                                               const float (&vs)[2]) {
  constexpr uint32_t kBad = kE5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;  // of a byte that is not finite
  uint32_t any = !(fabsf(vs[0]) <= FLT_MAX) || !(fabsf(vs[1]) <= FLT_MAX);
  if (mine)
#pragma unroll
    for (int w = 0; w < kDim / 16; ++w) {
      const uint4 v = *reinterpret_cast<const uint4*>(&x.v[lane][(w + lane) % (kDim / 16) * 16]);
      any |= __vcmpeq4(v.x & kBad, kBad) | __vcmpeq4(v.y & kBad, kBad) | __vcmpeq4(v.z & kBad, kBad) |
             __vcmpeq4(v.w & kBad, kBad);
    }
  return __any_sync(0xffffffffu, any != 0u);
}

// Then those values become 0 for the products; mark_not_finite does the rest when the item ends.
template <int kDim, bool kE5M2>
__device__ __forceinline__ void hide_not_finite(Stage<kDim>& x, bool mine, int lane, float (&vs)[2]) {
  constexpr uint32_t kBad = kE5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
  if (mine) {
    uint32_t* row = reinterpret_cast<uint32_t*>(x.v[lane]);
#pragma unroll 1
    for (int w = 0; w < kDim / 4; ++w) row[w] &= ~__vcmpeq4(row[w] & kBad, kBad);
  }
  if (!(fabsf(vs[0]) <= FLT_MAX)) vs[0] = 0.f;
  if (!(fabsf(vs[1]) <= FLT_MAX)) vs[1] = 0.f;
  fence_proxy_async_smem();  // the stage's next copy comes through another proxy
  __syncwarp();
}

// One tile; limit[i][r] - tok: how many of its tokens the lane's row r of
// fragment i sees (may be negative or past its end); least_limit: of the row that sees
// the fewest.  fresh: the item's first tile of this warp.  there: bit h where
// fragment h of the tile is; valid: its tokens that exist; ks, vs: the scales
// of its fragments.
template <int kDim, bool kE5M2, int kNR>
__device__ __forceinline__ void attend_tile(State<kDim> (&s)[kNR],
                                            const Stage<kDim>& x, const Queries<kDim> (&q)[kNR],
                                            const int (&limit)[kNR][2], int least_limit, int tok,
                                            uint32_t there, bool fresh, int valid,
                                            const float (&ks)[2], const float (&vs)[2], int lane) {
  const int g = lane / 4, t = lane % 4;
  float c[2][kNR][4] = {};
#pragma unroll
  for (int cc = 0; cc < kDim / 64; ++cc) {
    uint32_t k[2][2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 r = key_chunk(x, h, i, cc, g, t);
        k[h][i][0] = r.x;
        k[h][i][1] = r.y;
        k[h][i][2] = r.z;
        k[h][i][3] = r.w;
      }
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t k0 = k[h][0][w], k1 = k[h][1][w];
        const uint32_t a[4] = {
            f8x2_to_f16x2<kE5M2>(uint16_t(k0)), f8x2_to_f16x2<kE5M2>(uint16_t(k1)),
            f8x2_to_f16x2<kE5M2>(uint16_t(k0 >> 16)), f8x2_to_f16x2<kE5M2>(uint16_t(k1 >> 16))};
#pragma unroll
        for (int i = 0; i < kNR; ++i)
          mma_f16(c[h][i], a, q[i].b[4 * cc + w][0], q[i].b[4 * cc + w][1]);
      }
  }
  // scores in powers of two, less the running maximum; element 2e + r: token g + 8e, row r
  bool rises = fresh;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < kNR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[h][i][e] = fmaf(c[h][i][e], q[i].mul[e & 1] * ks[h], -s[i].m[e & 1]);
  if (tok + kTok > least_limit || there != 3u) {  // the same for the warp
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kNR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + 8 * (e >> 1) + kFrag * h + tok >= limit[i][e & 1] || !(there >> h & 1))
            c[h][i][e] = -INFINITY;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < kNR; ++i)
      rises |= fmaxf(fmaxf(c[h][i][0], c[h][i][1]), fmaxf(c[h][i][2], c[h][i][3])) > kLazy;
  if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
    for (int i = 0; i < kNR; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float up = fmaxf(fmaxf(c[0][i][r], c[0][i][2 + r]), fmaxf(c[1][i][r], c[1][i][2 + r]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
        // by how much the maximum rises: the first tile's sets it (m was 0), unless it is all
        // hidden -- tokens are seen from the first on, so then all of them are
        up = fresh ? (up == -INFINITY ? 0.f : up) : fmaxf(up, 0.f);
        const float shrink = exp2_fast(-up);
        s[i].m[r] += up;
        if (!fresh) {
          s[i].l[r] *= shrink;
#pragma unroll
          for (int j = 0; j < kDim / 16; ++j) {
            s[i].o[j][r] *= shrink;
            s[i].o[j][2 + r] *= shrink;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          c[h][i][r] -= up;
          c[h][i][2 + r] -= up;
        }
      }
  }
  uint32_t b[2][kNR][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < kNR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[h][i][e] = exp2_fast(c[h][i][e] + kLift);
        s[i].l[e & 1] += c[h][i][e];
      }
#pragma unroll
    for (int i = 0; i < kNR; ++i) {
      b[h][i][0] = transpose8x8(f16x2_bits(c[h][i][0], c[h][i][1]));
      b[h][i][1] = transpose8x8(f16x2_bits(c[h][i][2], c[h][i][3]));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[4][kDim / 32];
#pragma unroll
    for (int p = 0; p < 4; ++p) value_bytes(x, h, p, g, t, v[p]);
    if (valid < kTok || there != 3u) {  // what lies past the end may be anything: not even a 0 times it
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (kFrag * h + 2 * t + (p & 1) + 8 * (p >> 1) >= valid || !(there >> h & 1))
#pragma unroll
          for (int w = 0; w < kDim / 32; ++w) v[p][w] = 0u;
    }
#pragma unroll
    for (int j = 0; j < kDim / 16; ++j) {
      // bytes 2j and 2j + 1 of the four tokens: one matrix row each
      const uint32_t pick = (j & 1) ? 0x7362 : 0x5140;
      const uint32_t lo = __byte_perm(v[0][j / 2], v[1][j / 2], pick);
      const uint32_t hi = __byte_perm(v[2][j / 2], v[3][j / 2], pick);
      const uint32_t a[4] = {f8x2_to_f16x2<kE5M2>(uint16_t(lo)),
                             f8x2_to_f16x2<kE5M2>(uint16_t(lo >> 16)),
                             f8x2_to_f16x2<kE5M2>(uint16_t(hi)),
                             f8x2_to_f16x2<kE5M2>(uint16_t(hi >> 16))};
#pragma unroll
      for (int i = 0; i < kNR; ++i) {
        float d[4];
        mma_f16_new(d, a, b[h][i][0], b[h][i][1]);
        add_scaled4(s[i].o[j], vs[h] * kUnlift, d);
      }
    }
  }
}

// CTAs that fit on an SM: by shared memory at dim 128 (12 warps in all), by
// registers at dim 64.
constexpr int kMaxPerSm = 4;
constexpr int ctas_per_sm(int warps, int dim, int fragments) {
  return warps > 4 ? 1 : dim == 64 && fragments == 1 ? kMaxPerSm : 3;
}

__device__ __forceinline__ void add_scaled(float4& o, float& l, const float* v, float vl, float f) {
  l = fmaf(f, vl, l);
  o.x = fmaf(f, v[0], o.x);
  o.y = fmaf(f, v[1], o.y);
  o.z = fmaf(f, v[2], o.z);
  o.w = fmaf(f, v[3], o.w);
}

// Dimensions d .. d + 3 of a row: divided by its sum, zeros where it saw nothing.
template <int kDim>
__device__ __forceinline__ void write_out(const KvAttentionArgs& a, int t0, int head, int row, int d,
                                          const float4& o, float l) {
  const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
  __nv_bfloat16* out = a.O + (size_t(t0 + row / a.group) * a.heads * a.group + head * a.group +
                              row % a.group) * kDim + d;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(bf16x2_bits(o.x * inv, o.y * inv), bf16x2_bits(o.z * inv, o.w * inv));
}

// Row fragments that a CTA takes at a time: two (16 rows) read the cache half
// as often where a sequence may have more than 8 rows per cached head (131077 tokens, 16
// rows: 66 us with one, 55 with two); for up to 8 the second would be idle work (64
// sequences, 8 rows: 101 us with one, 112 with two).  More rows take further passes:
// the products bound those already (64 of up to 8192 tokens: 100 us for 8 rows, 208 for 32).
int row_fragments(const KvAttentionArgs& a) { return (long long)a.max_q * a.group > kRows ? 2 : 1; }

// Warps of a CTA.  With many items each SM has three CTAs of four, whose starts
// and joins of items overlap.  Where the SMs are at least twice the items, one CTA of
// twelve to an SM, each with a part of one item, leaves a third of the partials and
// lets an SM's warps end together (one sequence of 131077 tokens, 8 items: 70 us
// with four warps, 55 with twelve; 8 ragged ones of up to 16384, 64 items: 39 and
// 37).  Nearer to the SMs' number whole parts no longer fit ragged lengths (16 of up
// to 8192, 128 items: 35 us with four, 42 with twelve).
long long attention_items(const KvAttentionArgs& a) {
  const int rows = kRows * row_fragments(a);
  return ((long long)a.max_q * a.group + rows - 1) / rows * a.heads * a.B;
}
int attention_warps(const LaunchCtx& c, const KvAttentionArgs& a) {
  return 2 * attention_items(a) <= c.num_sms ? 12 : 4;
}

// CTAs: as many as run at once, or fewer where the tables cannot hold that much work.
int attention_grid(const LaunchCtx& c, const KvAttentionArgs& a) {
  const int warps = attention_warps(c, a);
  const long long tiles = max(1LL, ((long long)a.width * a.block + kTok - 1) / kTok);
  const long long items = attention_items(a);
  if (warps > 4) return int(min(items * ((tiles + kMinTiles - 1) / kMinTiles), (long long)c.num_sms));
  const int least = kMinTiles + kItemCost;
  const long long most = (items * (tiles + kItemCost) + least - 1) / least;
  return int(min(most, (long long)ctas_per_sm(warps, a.dim, row_fragments(a)) * c.num_sms));
}

// The counters' place does not depend on the call: what one call leaves there
// (zeros) is what the next one, of whatever size, finds.
size_t counter_bytes(const LaunchCtx& c) { return (size_t(kMaxPerSm) * c.num_sms * 4 + 255) / 256 * 256; }

// The flattened work of a call: items (sequence, row tile, cached head) in
// that order, each a run of tiles (behind what it costs).  A sequence with no
// cached token still has one tile per row tile and head, which writes zeros.
struct Sequence {
  int t0, n, len;      // first token on the packed axis, new tokens, cached tokens
  int row_tiles, tiles;  // tiles of each row tile and head
  long long total;       // with their items' costs
};

template <int kNR>
__device__ __forceinline__ Sequence sequence(const KvAttentionArgs& a, int b, int* status) {
  Sequence s;
  bool ok = sequence_tokens(a.cu, b, a.B, a.T, a.max_q, &s.t0, &s.n);
  if (!ok) s.n = 0;
  s.len = a.lens[b];
  if (s.len < 0 || (long long)s.len > (long long)a.width * a.block) {
    ok = false;
    s.len = 0;
  }
  if (!ok) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
  s.row_tiles = ceil_div(s.n * a.group, kRows * kNR);
  s.tiles = max(1, ceil_div(s.len, kTok));
  s.total = (long long)s.row_tiles * a.heads * (s.tiles + kItemCost);
  return s;
}

// Where a CTA is in its work.  It lies in shared memory, for what only the ends
// of an item need would crowd the registers of the loop between them.
struct Walk {
  long long u, u1;    // next and end of its run
  long long before;   // work of the sequences before b
  long long per;      // of a run
  int b;
  Sequence seq;
  int item, s0, s1;   // item in the sequence (row tile and head), tiles of it
  int first, last;    // CTAs that share it
};

// Outputs of an item that see a value, or a token of a block whose scale, that is not finite
// among its new tokens become NaN: by a look at those tokens' codes in the cache, into
// one warp's results.  Not inlined: few calls need it, and code that others have to jump
// over at the end of an item is fetched line by line (131077 tokens, 16 rows: 55 us so, 62 with
// the marks of those outputs kept in shared memory).
template <int kDim, bool kE5M2, int kR>
__device__ __noinline__ void mark_not_finite(const KvAttentionArgs& a, const Walk& w, float* so) {
  constexpr int kBad = kE5M2 ? 0x7c : 0x7f;
  const int head = w.item % a.heads, row0 = w.item / a.heads * kR;
  const int rows = w.seq.n * a.group, first_limit = w.seq.len - w.seq.n + 1;
  auto limit = [&](int r) { return row0 + r < rows ? first_limit + (row0 + r) / a.group : w.seq.len; };
  const int from = max(w.s0 * kTok, max(limit(0), 0) / kTok * kTok), to = min(w.s1 * kTok, w.seq.len);
  for (int tok = from + int(threadIdx.x) / 32; tok < to; tok += int(blockDim.x) / 32) {
    const int blk = a.table[size_t(w.b) * a.width + (tok >> a.log_block)];
    if (blk < 0 || blk >= a.num_blocks) continue;
    const size_t tile = size_t(blk) * a.heads + head;
    const uint8_t* v = a.vc + (tile * a.block + (tok & (a.block - 1))) * kDim;
    const bool scale = !(fabsf(a.vs[tile]) <= FLT_MAX);
    for (int d = threadIdx.x % 32; d < kDim; d += 32)
      if (scale || (v[d] & kBad) == kBad)
        for (int r = 0; r < kR; ++r)
          if (tok < limit(r)) so[r * (kDim + 4) + d] = NAN;
  }
}

// A partial result in the workspace: what a CTA knows of an item that it shares.
template <int kDim, int kNR>
struct Partial {
  float o[kRows * kNR][kDim];
  float m[kRows * kNR], l[kRows * kNR];
};

// Joins the partials of CTAs first .. last of one item, in that order.  What
// each one's rows have to be multiplied by comes first (in shared memory, kJoinMax
// CTAs at a time), so that the loads of the sums do not wait for one another.
constexpr int kJoinMax = 64;

template <int kDim, int kNR, int kWarps>
__device__ __forceinline__ void join_partials(const KvAttentionArgs& a,
                                              const Partial<kDim, kNR>* parts, int first, int last,
                                              int t0, int head, int row0, int rows, float* shared) {
  constexpr int kR = kRows * kNR;
  constexpr int kThreads = kWarps >= 8 && kR * kDim >= 1024 ? 256 : 128;  // the others only meet the barriers
  constexpr int kPer = kR * kDim / 4 / kThreads;
  static_assert(kPer * kThreads * 4 == kR * kDim, "a whole number for each thread");
  constexpr int kLanes = kThreads / kR;          // neighbouring lanes for each row's statistics
  const bool mine = threadIdx.x < kThreads;
  constexpr int kStep = kPer == 1 ? 16 : 32 / kPer;  // CTAs whose sums are in flight at once
  float* f = shared;                   // [kJoinMax][kR] factors
  float* ls = f + kJoinMax * kR;       // [kR] row sums
  float* shrink = ls + kR;             // [kR] of what was summed before
  const int r = threadIdx.x / kLanes % kR, q = threadIdx.x % kLanes;
  float m = kNone, l = 0.f;
  float4 o[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto part = [&](int c) -> const Partial<kDim, kNR>& { return parts[2 * c + (c == first ? 1 : 0)]; };
  for (int c0 = first; c0 <= last; c0 += kJoinMax) {
    const int n = min(kJoinMax, last + 1 - c0);
    constexpr int kMine = kJoinMax / kLanes;
    float pm[kMine], pl[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int c = mine ? q + i * kLanes : n;
      pm[i] = c < n ? __ldcg(&part(c0 + c).m[r]) : -INFINITY;
      pl[i] = c < n ? __ldcg(&part(c0 + c).l[r]) : 0.f;
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kMine; ++i) top = fmaxf(top, pm[i]);
#pragma unroll
    for (int x = 1; x < kLanes; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    __syncthreads();  // f is free
    const float s = exp2_fast(m - top);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const float e = exp2_fast(pm[i] - top);  // 0 past the last CTA
      sum = fmaf(e, pl[i], sum);
      if (mine) f[(q + i * kLanes) * kR + r] = e;
    }
#pragma unroll
    for (int x = 1; x < kLanes; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    m = top;
    l = fmaf(l, s, sum);
    if (mine && q == 0) {
      ls[r] = l;
      shrink[r] = s;
    }
    __syncthreads();
    if (!mine) continue;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float x = shrink[(threadIdx.x + kThreads * k) / (kDim / 4)];
      o[k] = make_float4(o[k].x * x, o[k].y * x, o[k].z * x, o[k].w * x);
    }
    for (int c = 0; c < n; c += kStep) {
      float4 v[kStep][kPer];
#pragma unroll
      for (int e = 0; e < kStep; ++e)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int i = threadIdx.x + kThreads * k;
          v[e][k] = c + e < n ? __ldcg(reinterpret_cast<const float4*>(
                                    &part(c0 + c + e).o[i / (kDim / 4)][i % (kDim / 4) * 4]))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int e = 0; e < kStep; ++e)
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const float x = f[min(c + e, kJoinMax - 1) * kR + (threadIdx.x + kThreads * k) / (kDim / 4)];
          o[k].x = fmaf(x, v[e][k].x, o[k].x);
          o[k].y = fmaf(x, v[e][k].y, o[k].y);
          o[k].z = fmaf(x, v[e][k].z, o[k].z);
          o[k].w = fmaf(x, v[e][k].w, o[k].w);
        }
    }
  }
  if (!mine) return;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = threadIdx.x + kThreads * k, row = i / (kDim / 4), d = i % (kDim / 4) * 4;
    if (row0 + row < rows) write_out<kDim>(a, t0, head, row0 + row, d, o[k], ls[row]);
  }
}

// The cache's codes as rows of dim bytes, in boxes of min(block, kTok) rows.
struct CacheMaps {
  CUtensorMap k, v;
};

// The CTAs share the work of all items evenly, in runs (or, where there are few
// items, in parts of one item each).  A CTA joins its
// warps' results in shared memory for each item of its run; an item that lies in
// several runs is joined from their partials, in CTA order, by whichever of
// them finishes last, so results do not depend on timing.
//   slot 2c      CTA c's share of an item that began before its run
//   slot 2c + 1  of an item that begins in its run and goes on
//   counter c    CTAs done with the item that goes on past CTA c's run (left at 0)
template <int kDim, bool kE5M2, int kNR, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, ctas_per_sm(kWarps, kDim, kNR))
    kv_attention_kernel(const __grid_constant__ KvAttentionArgs a,
                        const __grid_constant__ CacheMaps maps, int* counters,
                        Partial<kDim, kNR>* parts, int* status) {
  constexpr int kR = kRows * kNR;
  constexpr bool kWholeItems = kWarps > 4;
  extern __shared__ unsigned char raw[];
  unsigned char* shared = raw + (1024u - (smem_addr(raw) & 1023u)) % 1024u;
  float (*so)[kR][kDim + 4] = reinterpret_cast<float (*)[kR][kDim + 4]>(shared);
  __shared__ float sm[kWarps][kR], sl[kWarps][kR];
  __shared__ long long scan[kWarps];
  __shared__ Walk walks[2];  // the item's, and the next one's
  __shared__ int last_one;
  __shared__ int gave_up;  // a wait ran out
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ int not_finite;  // values of the item were hidden
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  Stage<kDim>* ring = reinterpret_cast<Stage<kDim>*>(shared) + warp * kStages;

  if (threadIdx.x == 0) {
    gave_up = not_finite = 0;
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&bars[0][i], 1);
    fence_mbar_init();
  }
  uint32_t phases = 0;     // bit s: the parity that stage s waits for next
  uint32_t in_flight = 0;  // bit s: it has been asked for

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  griddep_launch_dependents();
  griddep_wait();

  if constexpr (kWholeItems) {
    // One part of one item: the items in parts of `per` tiles, the fewest that
    // leaves no more parts than CTAs.  Thread b holds sequence b.
    Sequence seq = {};
    if (int(threadIdx.x) < a.B) seq = sequence<kNR>(a, threadIdx.x, status);
    const int items = seq.row_tiles * a.heads;
    auto cta_total = [&](long long v) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      __syncthreads();  // scan is free
      if (lane == 0) scan[warp] = v;
      __syncthreads();
      v = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += scan[w];
      return v;
    };
    const long long all = cta_total((long long)items * seq.tiles);
    int part = max(kMinTiles, int((all + gridDim.x - 1) / gridDim.x));
    int mine;
    long long parts_all;
    while (true) {  // ends: there are no more items than CTAs, and a part may be a whole one
      mine = items > 0 ? items * ceil_div(seq.tiles, part) : 0;
      parts_all = cta_total(mine);
      if (parts_all <= gridDim.x) break;
      part = max(part + 1, int(part * parts_all / gridDim.x));
    }
    if (blockIdx.x >= parts_all) return;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    for (int w = 0; w < warp; ++w) upto += int(scan[w]);
    if (int(blockIdx.x) < upto && int(blockIdx.x) >= upto - mine) {  // one thread's
      const int parts = ceil_div(seq.tiles, part), at = int(blockIdx.x) - (upto - mine);
      Walk w = {};
      w.u1 = 1;
      w.b = threadIdx.x;
      w.seq = seq;
      w.item = at / parts;
      w.s0 = at % parts * part;
      w.s1 = min(seq.tiles, w.s0 + part);
      w.first = int(blockIdx.x) - at % parts;
      w.last = w.first + parts - 1;
      walks[0] = w;
    }
  } else {
    // A run of the work of all items; a thread has a share of the sequences.
    const int per_thread = ceil_div(a.B, 32 * kWarps);
    const int b0 = min(a.B, int(threadIdx.x) * per_thread), b1 = min(a.B, b0 + per_thread);
    long long mine = 0;
    Sequence seq = {};
    for (int i = b0; i < b1; ++i) {
      seq = sequence<kNR>(a, i, status);
      mine += seq.total;
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) scan[warp] = upto;
    __syncthreads();
    long long U = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += scan[w];
      U += scan[w];
    }
    const long long per = max((long long)(kMinTiles + kItemCost), (U + gridDim.x - 1) / gridDim.x);
    const long long u0 = blockIdx.x * per, u1 = min(U, u0 + per);
    if (u0 >= u1) return;
    if (u0 >= upto - mine && u0 < upto) {  // one thread's
      long long at = upto - mine;
      int i = b0;
      if (b1 - b0 > 1)
        for (;; ++i) {
          seq = sequence<kNR>(a, i, status);
          if (u0 < at + seq.total) break;
          at += seq.total;
        }
      walks[0] = Walk{u0, u1, at, per, i, seq, 0, 0, 0, 0, 0};
    }
  }
  __syncthreads();

  for (int flip = 0; walks[flip].u < walks[flip].u1; flip ^= 1) {
    Walk w = walks[flip];
    if constexpr (kWholeItems) {
      w.u = w.u1;
    } else {
      while (w.u >= w.before + w.seq.total) {
        w.before += w.seq.total;
        w.seq = sequence<kNR>(a, ++w.b, status);
      }
      w.item = int((w.u - w.before) / (w.seq.tiles + kItemCost));
      const long long item0 = w.before + (long long)w.item * (w.seq.tiles + kItemCost) + kItemCost;
      w.s0 = int(max(w.u - item0, 0LL));
      w.s1 = int(min((long long)w.seq.tiles, w.u1 - item0));
      w.u = item0 + w.s1;
      if (w.s1 <= 0) break;  // the run ends within the item's cost
      w.first = int(item0 / w.per);
      w.last = int((item0 + w.seq.tiles - 1) / w.per);
    }
    if (threadIdx.x == 0) walks[flip ^ 1] = w;
    const int b = w.b, s0 = w.s0, s1 = w.s1;
    const Sequence q_seq = w.seq;
    const int head = w.item % a.heads, row0 = w.item / a.heads * kR;
    const int rows = q_seq.n * a.group, len = q_seq.len;

    // The warp takes tiles s0 + warp, s0 + warp + kWarps, ...: n_mine of them.
    const int n_mine = max(0, ceil_div(s1 - s0 - warp, kWarps));
    auto token_of = [&](int i) { return (s0 + warp + i * kWarps) * kTok; };
    // Where they lie.  Lane l looks up the l-th of 32 at a time: the
    // cache row of each fragment's first token (-1: not there) and its scales, for
    // the batch in use and, while that is worked on, the one after it.
    const int* table = a.table + size_t(b) * a.width;
    const bool halves = a.block < kTok;  // a tile lies in two blocks
    struct Batch {
      int row[2];
      float k[2], v[2];
    } batch = {}, after = {};
    auto look_up = [&](Batch& x, int i) {
      const int tok = token_of(i);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = tok + kFrag * h;
        x.row[h] = -1;
        if (h == 1 && !halves) {
          x.row[1] = x.row[0] < 0 ? -1 : x.row[0] + kFrag;
        } else if (i < n_mine && at < len) {
          const int blk = table[at >> a.log_block];
          if (blk >= 0 && blk < a.num_blocks)
            x.row[h] = ((blk * a.heads + head) << a.log_block) + (at & (a.block - 1));
          else  // a bad table entry: its tokens count as not there
            raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
        }
      }
    };
    auto look_up_scales = [&](Batch& x) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !halves) {
          x.k[1] = x.k[0];
          x.v[1] = x.v[0];
        } else {
          x.k[h] = x.row[h] < 0 ? 0.f : a.ks[x.row[h] >> a.log_block];
          x.v[h] = x.row[h] < 0 ? 0.f : a.vs[x.row[h] >> a.log_block];
        }
      }
    };
    auto fetch = [&](int stage, const Batch& x, int l) {
      int row[2];
      row[0] = __shfl_sync(0xffffffffu, x.row[0], l);
      row[1] = __shfl_sync(0xffffffffu, x.row[1], l);
      if (row[0] < 0 && row[1] < 0) return;
      in_flight |= 1u << stage;
      if (lane != 0) return;
      constexpr int kHalf = kFrag * kDim;
      uint64_t* bar = &bars[warp][stage];
      mbar_arrive_expect_tx(bar, 2 * kHalf * (int(row[0] >= 0) + int(row[1] >= 0)));
      if (!halves) {
        tma_load_2d(ring[stage].k, &maps.k, bar, 0, row[0]);
        tma_load_2d(ring[stage].v, &maps.v, bar, 0, row[0]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (row[h] < 0) continue;
          tma_load_2d(ring[stage].k[kFrag * h], &maps.k, bar, 0, row[h]);
          tma_load_2d(ring[stage].v[kFrag * h], &maps.v, bar, 0, row[h]);
        }
      }
    };
    look_up(batch, lane);
    // Queries and scales are asked for before the tiles: behind the first tiles of all
    // warps (29 MB) they would come microseconds late.
    RawQuery<kDim> raw_q[kNR];
#pragma unroll
    for (int i = 0; i < kNR; ++i) {
      const int row = row0 + kRows * i + g;  // whose query this lane loads
      raw_q[i] = load_query<kDim>(row < rows ? a.Q + (q_seq.t0 + row / a.group) * a.ld_q +
                                                   (head * a.group + row % a.group) * kDim
                                             : nullptr, t);
    }
    look_up_scales(batch);
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i, batch, i);
    look_up(after, 32 + lane);
    Queries<kDim> q[kNR];
    State<kDim> s[kNR];
    int limit[kNR][2];  // tokens that the lane's rows see
#pragma unroll
    for (int i = 0; i < kNR; ++i) {
      take_queries<kDim>(q[i], raw_q[i], a.scale * 1.44269504088896341f, t);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int rr = row0 + kRows * i + 2 * t + r;
        limit[i][r] = rr < rows ? len - q_seq.n + 1 + rr / a.group : len;
      }
      clear(s[i]);
    }
    const int least_limit = len - q_seq.n + 1 + row0 / a.group;
    int stage = 0;
    bool fresh = true;
    for (int i = 0; i < n_mine; ++i) {
      const int l = i & 31;
      if (l == 16) look_up_scales(after);
      const uint32_t there = uint32_t(__shfl_sync(0xffffffffu, batch.row[0], l) >= 0) |
                             uint32_t(__shfl_sync(0xffffffffu, batch.row[1], l) >= 0) << 1;
      if (there != 0) {
        const int tok = token_of(i);
        float ks[2], vs[2];
        ks[0] = ks[1] = __shfl_sync(0xffffffffu, batch.k[0], l);
        vs[0] = vs[1] = __shfl_sync(0xffffffffu, batch.v[0], l);
        if (halves) {
          ks[1] = __shfl_sync(0xffffffffu, batch.k[1], l);
          vs[1] = __shfl_sync(0xffffffffu, batch.v[1], l);
        }
        // one outcome for the warp: what follows is warp-wide
        if (!__all_sync(0xffffffffu, mbar_wait_within(&bars[warp][stage], phases >> stage & 1,
                                                      &gave_up, a.wait_ns))) {
          // results are void; what is still in flight lands before the CTA ends
          gave_up = 1;
          raise_status(status, FP8GEMM_ERR_TIMEOUT);
          for (int k = 0; k < kStages; ++k)
            if (in_flight >> k & 1) mbar_drain(&bars[warp][k], phases >> k & 1);
          break;
        }
        phases ^= 1u << stage;
        in_flight &= ~(1u << stage);
        if (tok + kTok > least_limit && least_limit < len) {  // the same for the warp
          const bool mine = tok + lane >= least_limit && tok + lane < len && (there >> (lane / kFrag) & 1);
          if (any_not_finite<kDim, kE5M2>(ring[stage], mine, lane, vs)) {
            hide_not_finite<kDim, kE5M2>(ring[stage], mine, lane, vs);
            not_finite = 1;
          }
        }
        attend_tile<kDim, kE5M2, kNR>(s, ring[stage], q, limit, least_limit, tok, there, fresh,
                                      len - tok, ks, vs, lane);
        fresh = false;
        __syncwarp();  // the stage has been read
      }
      if (l + kStages < 32)
        fetch(stage, batch, l + kStages);
      else
        fetch(stage, after, l + kStages - 32);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (l == 31) {
        batch = after;
        look_up(after, i + 33 + lane);
      }
    }
    __syncthreads();  // the rings become the place to join the warps' results
    if (gave_up) break;

#pragma unroll
    for (int i = 0; i < kNR; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = kRows * i + 2 * t + r;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s[i].l[r] += __shfl_xor_sync(0xffffffffu, s[i].l[r], o);
        if (g == 0) {
          sm[warp][row] = s[i].l[r] == 0.f ? kNone : s[i].m[r];
          sl[warp][row] = s[i].l[r] * kUnlift;
        }
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j)
          *reinterpret_cast<float2*>(&so[warp][row][g * (kDim / 8) + 2 * j]) =
              make_float2(s[i].o[j][r], s[i].o[j][2 + r]);
      }
    __syncthreads();
    const Walk& done = walks[flip ^ 1];
    if (not_finite) {
      mark_not_finite<kDim, kE5M2, kR>(a, done, &so[0][0][0]);
      __syncthreads();
      if (threadIdx.x == 0) not_finite = 0;
    }
    const bool begins = done.s0 == 0, ends = done.s1 == done.seq.tiles;
    const int out_head = done.item % a.heads, out_row0 = done.item / a.heads * kR;
    const int out_rows = done.seq.n * a.group;
    Partial<kDim, kNR>* part = parts + 2 * blockIdx.x + (begins ? 1 : 0);
    for (int i = threadIdx.x; i < kR * kDim / 4; i += 32 * kWarps) {
      const int r = i / (kDim / 4), d = i % (kDim / 4) * 4, row = out_row0 + r;
      float m = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) add_scaled(o, l, so[w][r] + d, sl[w][r], exp2_fast(sm[w][r] - m));
      if (begins && ends) {
        if (row < out_rows) write_out<kDim>(a, done.seq.t0, out_head, row, d, o, l);
      } else {
        *reinterpret_cast<float4*>(&part->o[r][d]) = o;
        if (d == 0) {
          part->m[r] = m;
          part->l[r] = l;
        }
      }
    }
    fence_proxy_async_smem();  // the copies that follow come through another proxy
    __syncthreads();           // the shared buffers are free, and this CTA's partial is written
    if (!(begins && ends)) {
      if (threadIdx.x == 0) last_one = atomic_add_acq_rel_gpu(counters + done.first, 1) == done.last - done.first;
      __syncthreads();
      if (last_one) {
        if (threadIdx.x == 0) counters[done.first] = 0;
        join_partials<kDim, kNR, kWarps>(a, parts, done.first, done.last, done.seq.t0, out_head,
                                         out_row0, out_rows,
                                 reinterpret_cast<float*>(shared));
        fence_proxy_async_smem();
        __syncthreads();
      }
    }
  }
}

template <int kDim, bool kE5M2, int kNR, int kWarps>
cudaError_t launch(const LaunchCtx& c, const KvAttentionArgs& a, const CacheMaps& maps, void* ws) {
  const int grid = attention_grid(c, a);
  int* counters = static_cast<int*>(ws);
  auto* parts = reinterpret_cast<Partial<kDim, kNR>*>(static_cast<char*>(ws) + counter_bytes(c));
  constexpr size_t kRings = sizeof(Stage<kDim>) * kStages * kWarps;
  constexpr size_t kJoin = sizeof(float) * kWarps * kRows * kNR * (kDim + 4);
  constexpr size_t kFactors = sizeof(float) * (kJoinMax + 2) * kRows * kNR;
  constexpr size_t kMore = kJoin > kFactors ? kJoin : kFactors;
  constexpr size_t kSmem = 1024 + (kRings > kMore ? kRings : kMore);
  auto fn = kv_attention_kernel<kDim, kE5M2, kNR, kWarps>;
  static SmemLimit limit;
  if (cudaError_t e = limit.raise(c, reinterpret_cast<const void*>(fn), kSmem)) return e;
  return launch_dependent(c, fn, grid, 32 * kWarps, kSmem, a, maps, counters, parts, c.status);
}

template <int kNR, int kWarps>
cudaError_t launch_shape(const LaunchCtx& c, const KvAttentionArgs& a, const CacheMaps& maps, void* ws) {
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  if (a.dim == 128)
    return e5 ? launch<128, true, kNR, kWarps>(c, a, maps, ws) : launch<128, false, kNR, kWarps>(c, a, maps, ws);
  return e5 ? launch<64, true, kNR, kWarps>(c, a, maps, ws) : launch<64, false, kNR, kWarps>(c, a, maps, ws);
}

}  // namespace

// Two partials for each CTA of the widest variant, for every call alike: a
// stream's buffer stays where it is (a captured graph holds its address).
size_t kv_attention_workspace_bytes(const LaunchCtx& c) {
  constexpr size_t kWide = ctas_per_sm(4, 128, 2) * sizeof(Partial<128, 2>);
  constexpr size_t kNarrow = ctas_per_sm(4, 64, 1) * sizeof(Partial<64, 1>);
  return counter_bytes(c) + 2 * c.num_sms * (kWide > kNarrow ? kWide : kNarrow);
}

cudaError_t launch_kv_attention(const LaunchCtx& c, const KvAttentionArgs& a, void* ws) {
  CacheMaps maps;
  const uint64_t rows = max(uint64_t(a.num_blocks) * a.heads * a.block, uint64_t(1));
  const uint32_t box = min(a.block, kTok);
  if (!make_tmap_rows(&maps.k, a.kc, rows, a.dim, box) || !make_tmap_rows(&maps.v, a.vc, rows, a.dim, box))
    return cudaErrorInvalidValue;
  if (attention_warps(c, a) == 12)
    return row_fragments(a) == 1 ? launch_shape<1, 12>(c, a, maps, ws) : launch_shape<2, 12>(c, a, maps, ws);
  return row_fragments(a) == 1 ? launch_shape<1, 4>(c, a, maps, ws) : launch_shape<2, 4>(c, a, maps, ws);
}

}  // namespace fp8gemm
