// kv_attention.cu -- attention of a sequence's newest tokens over its paged
// FP8 cache (kv_cache.cu has the layout).
//
//   o = sum_j p_j v_j,  p = softmax over the visible j of (scale q . k_j)
//
// The query of new token i of n sees the first len - n + 1 + i cached tokens
// (its own among them); a row that sees none gives zeros.  Query heads h g ..
// h g + g - 1 read the cached head h, so their rows share every byte of it.
//
// Bound by the cache's bytes: each is read once and straight into the
// registers of the tensor-core fragment it belongs to, with no pass through
// shared memory.  Both products are taken transposed so that tokens (and the
// head's dimension) fill the 16-row side of m16n8k16 and 8 query rows the other:
//   S^T [16 tokens, 8 rows] = K [16, dim] Q^T      O^T [dim, 8 rows] += V^T [dim, 16] P^T
// The order of a contraction is free, so the dimension is dealt to the
// fragment's k index such that a lane's share of a key is 16 neighbouring bytes, and the
// output dimension to V^T's rows such that a lane's share of a value is too.
// FP8 codes are exact in FP16; q is shifted by a power of two per row to use
// FP16's range (BF16 has fewer mantissa bits); p is rounded to FP16 (11
// bits, far below the BF16 output's step).  Scores, statistics, sums and the
// output accumulate in FP32; a tile's scales are applied to its FP32 products.
#include "common.cuh"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kTok = 16;   // tokens per tile: one fragment
constexpr int kRows = 8;   // query rows per fragment
constexpr int kWarps = 4;
constexpr int kUnit = kWarps * kTok;  // tokens of a unit: a tile for each warp
constexpr int kMinUnits = 4;  // a CTA's least share: fewer would cost more to join than to do
constexpr float kLazy = 8.f;  // the running maximum may lag by 2^8: p stays below 256

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

// Cache bytes: read once, so not kept in L1.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// A lane's share of 16 tokens of one head.  With lane = 4 g + t:
//   keys    tokens g and g + 8, bytes 64 c + 16 t .. + 15
//   values  tokens 2t, 2t + 1, 2t + 8, 2t + 9, bytes (dim / 8) g .. + dim / 8 - 1
template <int kDim>
struct Tile {
  uint32_t k[2][kDim / 64][4];
  uint32_t v[4][kDim / 32];
  float ks, vs;
  bool there;
};

// Tokens at and past `valid` read as zeros, whatever the cache holds there.
template <int kDim>
__device__ __forceinline__ void load_tile(Tile<kDim>& x, const uint8_t* k, const uint8_t* v,
                                          int valid, int g, int t) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int c = 0; c < kDim / 64; ++c) {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (g + 8 * i < valid) r = ld_stream16(k + (g + 8 * i) * kDim + 64 * c + 16 * t);
      x.k[i][c][0] = r.x;
      x.k[i][c][1] = r.y;
      x.k[i][c][2] = r.z;
      x.k[i][c][3] = r.w;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = 2 * t + (i & 1) + 8 * (i >> 1);
    const uint8_t* p = v + tok * kDim + g * (kDim / 8);
    if constexpr (kDim == 128) {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (tok < valid) r = ld_stream16(p);
      x.v[i][0] = r.x;
      x.v[i][1] = r.y;
      x.v[i][2] = r.z;
      x.v[i][3] = r.w;
    } else {
      uint2 r = make_uint2(0, 0);
      if (tok < valid) r = ld_stream8(p);
      x.v[i][0] = r.x;
      x.v[i][1] = r.y;
    }
  }
}

// The queries of 8 rows as the k16 x n8 fragments that match Tile's keys, and
// what their products have to be multiplied by (rows 2t and 2t + 1 of this lane).
template <int kDim>
struct Queries {
  uint32_t b[kDim / 16][2];
  float mul[2];
};

template <int kDim>
__device__ __forceinline__ void load_queries(Queries<kDim>& q, const __nv_bfloat16* row,
                                             float scale_log2, int t) {
  float x[kDim / 64][16];
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < kDim / 64; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      Raw8<__nv_bfloat16> r;
      zero8(r);
      if (row) r = load8(row + 64 * c + 16 * t + 8 * e);
      float f[8];
      unpack8(r, f);
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

// Running softmax of a lane's two rows and its share of O^T: o[j] holds
// dimensions (dim/8) g + 2j (rows 2t, 2t + 1) and + 1 (rows 2t, 2t + 1).
template <int kDim>
struct State {
  float m[2], l[2];  // l: this lane's tokens only
  float o[kDim / 16][4];
};

template <int kDim>
__device__ __forceinline__ void clear(State<kDim>& s) {
  s.m[0] = s.m[1] = -INFINITY;
  s.l[0] = s.l[1] = 0.f;
#pragma unroll
  for (int j = 0; j < kDim / 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s.o[j][e] = 0.f;
}

// One tile; sees[r]: how many of its tokens the lane's row r sees (may be
// negative or past 16).
template <int kDim, bool kE5M2>
__device__ __forceinline__ void attend_tile(State<kDim>& s, const Tile<kDim>& x,
                                            const Queries<kDim>& q, const int (&sees)[2], int g) {
  float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < kDim / 16; ++ks) {
    const uint32_t k0 = x.k[0][ks / 4][ks % 4], k1 = x.k[1][ks / 4][ks % 4];
    const uint32_t a[4] = {f8x2_to_f16x2<kE5M2>(uint16_t(k0)), f8x2_to_f16x2<kE5M2>(uint16_t(k1)),
                           f8x2_to_f16x2<kE5M2>(uint16_t(k0 >> 16)),
                           f8x2_to_f16x2<kE5M2>(uint16_t(k1 >> 16))};
    mma_f16(c, a, q.b[ks][0], q.b[ks][1]);
  }
  // scores in powers of two; element 2i + r: token g + 8i, row r
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c[e] = c[e] * (q.mul[e & 1] * x.ks);
    if (g + 8 * (e >> 1) >= sees[e & 1]) c[e] = -INFINITY;
  }
  const float top0 = fmaxf(c[0], c[2]), top1 = fmaxf(c[1], c[3]);
  if (__any_sync(0xffffffffu, top0 > s.m[0] + kLazy || top1 > s.m[1] + kLazy)) {
    float top[2] = {top0, top1};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
      const float m = fmaxf(s.m[r], top[r]);
      const float shrink = m == -INFINITY ? 1.f : exp2f(s.m[r] - m);
      s.m[r] = m;
      s.l[r] *= shrink;
#pragma unroll
      for (int j = 0; j < kDim / 16; ++j) {
        s.o[j][r] *= shrink;
        s.o[j][2 + r] *= shrink;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float m = s.m[e & 1];
    c[e] = exp2f(c[e] - (m == -INFINITY ? 0.f : m));
    s.l[e & 1] += c[e];
  }
  const uint32_t b0 = transpose8x8(f16x2_bits(c[0], c[1]));
  const uint32_t b1 = transpose8x8(f16x2_bits(c[2], c[3]));
#pragma unroll
  for (int j = 0; j < kDim / 16; ++j) {
    // bytes 2j and 2j + 1 of the four tokens: one matrix row each
    const uint32_t pick = (j & 1) ? 0x7362 : 0x5140;
    const uint32_t lo = __byte_perm(x.v[0][j / 2], x.v[1][j / 2], pick);
    const uint32_t hi = __byte_perm(x.v[2][j / 2], x.v[3][j / 2], pick);
    const uint32_t a[4] = {f8x2_to_f16x2<kE5M2>(uint16_t(lo)),
                           f8x2_to_f16x2<kE5M2>(uint16_t(lo >> 16)),
                           f8x2_to_f16x2<kE5M2>(uint16_t(hi)),
                           f8x2_to_f16x2<kE5M2>(uint16_t(hi >> 16))};
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    mma_f16(d, a, b0, b1);
#pragma unroll
    for (int e = 0; e < 4; ++e) s.o[j][e] = fmaf(d[e], x.vs, s.o[j][e]);
  }
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
// as often where a sequence may have more than 8 rows per cached head.
int row_fragments(const KvAttentionArgs& a) { return (long long)a.max_q * a.group > kRows ? 2 : 1; }

// CTAs that fit on an SM by their registers (168 a thread at dim 128 and one
// fragment, 255 with two; 128 and 168 at dim 64).
constexpr int kMaxPerSm = 4;
int ctas_per_sm(const KvAttentionArgs& a) { return (a.dim == 64 ? 4 : 3) - (row_fragments(a) - 1); }

// CTAs: as many as run at once, or fewer where the tables cannot hold that much work.
int attention_grid(const LaunchCtx& c, const KvAttentionArgs& a) {
  const long long row_tiles = ((long long)a.max_q * a.group + kRows * row_fragments(a) - 1) /
                              (kRows * row_fragments(a));
  const long long units = max(1LL, ((long long)a.width * a.block + kUnit - 1) / kUnit);
  const long long most = (row_tiles * a.heads * a.B * units + kMinUnits - 1) / kMinUnits;
  return int(min(most, (long long)ctas_per_sm(a) * c.num_sms));
}

// The counters' place does not depend on the call: what one call leaves there
// (zeros) is what the next one, of whatever size, finds.
size_t counter_bytes(const LaunchCtx& c) { return (size_t(kMaxPerSm) * c.num_sms * 4 + 255) / 256 * 256; }


// The flattened work of a call: items (sequence, row tile, cached head) in
// that order, each a run of units.  A sequence with no
// cached token still has one unit per row tile and head, which writes zeros.
struct Sequence {
  int t0, n, len;      // first token on the packed axis, new tokens, cached tokens
  int row_tiles, units;  // per row tile and head
  long long total;
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
  s.units = max(1, ceil_div(s.len, kUnit));
  s.total = (long long)s.row_tiles * a.heads * s.units;
  return s;
}

// Where a unit lies: its sequence and what is before that, found by the whole CTA.
struct Place {
  int b;
  long long before;  // units of the sequences before b
};

// A partial result in the workspace: what a CTA knows of an item that it shares.
template <int kDim, int kNR>
struct Partial {
  float o[kRows * kNR][kDim];
  float m[kRows * kNR], l[kRows * kNR];
};

// The CTAs share the units of all items evenly, in runs.  A CTA joins its
// warps' results in shared memory for each item of its run; an item that lies in
// several runs is joined from their partials, in CTA order, by whichever of
// them finishes last, so results do not depend on timing.
//   slot 2c      CTA c's share of an item that began before its run
//   slot 2c + 1  of an item that begins in its run and goes on
//   counter c    CTAs done with the item that goes on past CTA c's run (left at 0)
template <int kDim, bool kE5M2, int kNR>
__global__ void __launch_bounds__(32 * kWarps) kv_attention_kernel(const KvAttentionArgs a,
                                                                   int* counters,
                                                                   Partial<kDim, kNR>* parts,
                                                                   int* status) {
  constexpr int kR = kRows * kNR;
  __shared__ float so[kWarps][kR][kDim + 4];
  __shared__ float sm[kWarps][kR], sl[kWarps][kR];
  __shared__ long long scan[kWarps];
  __shared__ Place place;
  __shared__ int last_one;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;

  // all units, and each thread's share of the sequences
  const int per_thread = ceil_div(a.B, 32 * kWarps);
  const int b0 = min(a.B, int(threadIdx.x) * per_thread), b1 = min(a.B, b0 + per_thread);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += sequence<kNR>(a, b, status).total;
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
  const long long per = max((long long)kMinUnits, (U + gridDim.x - 1) / gridDim.x);
  const long long u0 = blockIdx.x * per, u1 = min(U, u0 + per);
  if (u0 >= u1) return;
  if (u0 >= upto - mine && u0 < upto) {  // one thread's
    long long before = upto - mine;
    for (int b = b0; b < b1; ++b) {
      const long long n = sequence<kNR>(a, b, status).total;
      if (u0 < before + n) {
        place = Place{b, before};
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  int b = place.b;
  long long before = place.before;
  Sequence q_seq = sequence<kNR>(a, b, status);

  for (long long u = u0; u < u1;) {
    while (u >= before + q_seq.total) {
      before += q_seq.total;
      q_seq = sequence<kNR>(a, ++b, status);
    }
    const int item = int((u - before) / q_seq.units);  // row tile and head
    const long long item0 = before + (long long)item * q_seq.units;
    const int head = item % a.heads, row0 = item / a.heads * kR;
    const int s0 = int(u - item0), s1 = int(min((long long)q_seq.units, u1 - item0));
    const int rows = q_seq.n * a.group, len = q_seq.len;

    Queries<kDim> q[kNR];
    State<kDim> s[kNR];
    int limit[kNR][2];  // tokens that the lane's rows see
#pragma unroll
    for (int i = 0; i < kNR; ++i) {
      const int row = row0 + kRows * i + g;  // whose query this lane loads
      const __nv_bfloat16* p =
          row < rows ? a.Q + (q_seq.t0 + row / a.group) * a.ld_q +
                           (head * a.group + row % a.group) * kDim
                     : nullptr;
      load_queries<kDim>(q[i], p, a.scale * 1.44269504088896341f, t);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int rr = row0 + kRows * i + 2 * t + r;
        limit[i][r] = rr < rows ? len - q_seq.n + 1 + rr / a.group : 0;
      }
      clear(s[i]);
    }
    // two tiles in flight: the next one's bytes are asked for before this one is used
    Tile<kDim> x[2];
    auto fetch = [&](Tile<kDim>& d, int unit) {
      const int tok = unit * kUnit + warp * kTok;
      const int blk = tok < len ? a.table[size_t(b) * a.width + tok / a.block] : -1;
      const bool there = blk >= 0 && blk < a.num_blocks;
      if (tok < len && !there && lane == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
      const size_t tile = there ? size_t(blk) * a.heads + head : 0;
      const size_t at = there ? (tile * a.block + tok % a.block) * kDim : 0;
      load_tile<kDim>(d, a.kc + at, a.vc + at, there ? len - tok : 0, g, t);
      d.ks = there ? a.ks[tile] : 0.f;
      d.vs = there ? a.vs[tile] : 0.f;
      d.there = there;
    };
    auto use = [&](const Tile<kDim>& d, int unit) {
      if (!d.there) return;  // past the end, or a bad table entry: counts as not there
      const int tok = unit * kUnit + warp * kTok;
#pragma unroll
      for (int i = 0; i < kNR; ++i) {
        const int sees[2] = {limit[i][0] - tok, limit[i][1] - tok};
        attend_tile<kDim, kE5M2>(s[i], d, q[i], sees, g);
      }
    };
    fetch(x[0], s0);
    for (int i = s0; i < s1; i += 2) {
      if (i + 1 < s1) fetch(x[1], i + 1);
      use(x[0], i);
      if (i + 2 < s1) fetch(x[0], i + 2);
      if (i + 1 < s1) use(x[1], i + 1);
    }

#pragma unroll
    for (int i = 0; i < kNR; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = kRows * i + 2 * t + r;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s[i].l[r] += __shfl_xor_sync(0xffffffffu, s[i].l[r], o);
        if (g == 0) {
          sm[warp][row] = s[i].m[r];
          sl[warp][row] = s[i].l[r];
        }
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j)
          *reinterpret_cast<float2*>(&so[warp][row][g * (kDim / 8) + 2 * j]) =
              make_float2(s[i].o[j][r], s[i].o[j][2 + r]);
      }
    __syncthreads();
    const bool begins = s0 == 0, ends = s1 == q_seq.units;
    const int first = int(item0 / per), last = int((item0 + q_seq.units - 1) / per);
    Partial<kDim, kNR>* part = parts + 2 * blockIdx.x + (begins ? 1 : 0);
    for (int i = threadIdx.x; i < kR * kDim / 4; i += 32 * kWarps) {
      const int r = i / (kDim / 4), d = i % (kDim / 4) * 4, row = row0 + r;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) add_scaled(o, l, so[w][r] + d, sl[w][r], exp2f(sm[w][r] - m));
      }
      if (begins && ends) {
        if (row < rows) write_out<kDim>(a, q_seq.t0, head, row, d, o, l);
      } else {
        *reinterpret_cast<float4*>(&part->o[r][d]) = o;
        if (d == 0) {
          part->m[r] = m;
          part->l[r] = l;
        }
      }
    }
    __syncthreads();  // the shared buffers are free, and this CTA's partial is written
    if (!(begins && ends)) {
      if (threadIdx.x == 0) last_one = atomic_add_acq_rel_gpu(counters + first, 1) == last - first;
      __syncthreads();
      if (last_one) {
        if (threadIdx.x == 0) counters[first] = 0;
        for (int i = threadIdx.x; i < kR * kDim / 4; i += 32 * kWarps) {
          const int r = i / (kDim / 4), d = i % (kDim / 4) * 4, row = row0 + r;
          if (row >= rows) continue;
          float m = -INFINITY;
          for (int c = first; c <= last; ++c)
            m = fmaxf(m, __ldcg(&parts[2 * c + (c == first ? 1 : 0)].m[r]));
          float l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          if (m != -INFINITY) {
            for (int c = first; c <= last; ++c) {
              const Partial<kDim, kNR>& p = parts[2 * c + (c == first ? 1 : 0)];
              const float4 v = __ldcg(reinterpret_cast<const float4*>(&p.o[r][d]));
              add_scaled(o, l, &v.x, __ldcg(&p.l[r]), exp2f(__ldcg(&p.m[r]) - m));
            }
          }
          write_out<kDim>(a, q_seq.t0, head, row, d, o, l);
        }
      }
    }
    u = item0 + s1;
  }
}

template <int kDim, bool kE5M2, int kNR>
cudaError_t launch(const LaunchCtx& c, const KvAttentionArgs& a, void* ws) {
  const int grid = attention_grid(c, a);
  int* counters = static_cast<int*>(ws);
  auto* parts = reinterpret_cast<Partial<kDim, kNR>*>(static_cast<char*>(ws) + counter_bytes(c));
  kv_attention_kernel<kDim, kE5M2, kNR><<<grid, 32 * kWarps, 0, c.stream>>>(a, counters, parts, c.status);
  return cudaGetLastError();
}

template <int kNR>
cudaError_t launch_rows(const LaunchCtx& c, const KvAttentionArgs& a, void* ws) {
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  if (a.dim == 128) return e5 ? launch<128, true, kNR>(c, a, ws) : launch<128, false, kNR>(c, a, ws);
  return e5 ? launch<64, true, kNR>(c, a, ws) : launch<64, false, kNR>(c, a, ws);
}

}  // namespace

size_t kv_attention_workspace_bytes(const LaunchCtx& c, const KvAttentionArgs& a) {
  const int grid = attention_grid(c, a);
  return counter_bytes(c) + size_t(2) * grid * row_fragments(a) * kRows * (a.dim + 2) * 4;
}

cudaError_t launch_kv_attention(const LaunchCtx& c, const KvAttentionArgs& a, void* ws) {
  return row_fragments(a) == 1 ? launch_rows<1>(c, a, ws) : launch_rows<2>(c, a, ws);
}

}  // namespace fp8gemm
