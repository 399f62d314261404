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

// Grid (row tiles, heads, B): the CTA's warps share the tiles of one sequence
// and head, every kWarps-th each, and are joined in shared memory.
template <int kDim, bool kE5M2>
__global__ void __launch_bounds__(32 * kWarps) kv_attention_kernel(const KvAttentionArgs a,
                                                                   int* status) {
  __shared__ float so[kWarps][kRows][kDim];
  __shared__ float sm[kWarps][kRows], sl[kWarps][kRows];
  const int b = blockIdx.z, head = blockIdx.y;
  int t0 = 0, n = 0;
  if (!sequence_tokens(a.cu, b, a.B, a.T, a.max_q, &t0, &n)) {
    if (threadIdx.x == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    return;
  }
  const int row0 = blockIdx.x * kRows, rows = n * a.group;
  if (row0 >= rows) return;
  int len = a.lens[b];
  if (len < 0 || (long long)len > (long long)a.width * a.block) {
    if (threadIdx.x == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
    len = 0;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;

  Queries<kDim> q;
  const int mine = row0 + g;  // the row whose query this lane loads
  const __nv_bfloat16* qrow =
      mine < rows ? a.Q + (t0 + mine / a.group) * a.ld_q + (head * a.group + mine % a.group) * kDim
                  : nullptr;
  load_queries<kDim>(q, qrow, a.scale * 1.44269504088896341f, t);
  int limit[2];  // tokens that rows 2t and 2t + 1 see
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row0 + 2 * t + r;
    limit[r] = row < rows ? len - n + 1 + row / a.group : 0;
  }
  State<kDim> s;
  clear(s);
  for (int tok = warp * kTok; tok < len; tok += kWarps * kTok) {
    const int blk = a.table[size_t(b) * a.width + tok / a.block];
    if (blk < 0 || blk >= a.num_blocks) {  // the tile counts as not there
      if (lane == 0) raise_status(status, FP8GEMM_ERR_DEVICE_STATUS);
      continue;
    }
    const size_t tile = size_t(blk) * a.heads + head;
    const size_t at = (tile * a.block + tok % a.block) * kDim;
    Tile<kDim> x;
    load_tile<kDim>(x, a.kc + at, a.vc + at, len - tok, g, t);
    x.ks = a.ks[tile];
    x.vs = a.vs[tile];
    const int sees[2] = {limit[0] - tok, limit[1] - tok};
    attend_tile<kDim, kE5M2>(s, x, q, sees, g);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) s.l[r] += __shfl_xor_sync(0xffffffffu, s.l[r], o);
    if (g == 0) {
      sm[warp][2 * t + r] = s.m[r];
      sl[warp][2 * t + r] = s.l[r];
    }
#pragma unroll
    for (int j = 0; j < kDim / 16; ++j) {
      so[warp][2 * t + r][g * (kDim / 8) + 2 * j] = s.o[j][r];
      so[warp][2 * t + r][g * (kDim / 8) + 2 * j + 1] = s.o[j][2 + r];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kDim / 2; i += 32 * kWarps) {
    const int r = i / (kDim / 2), d = i % (kDim / 2) * 2;
    if (row0 + r >= rows) break;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
    if (m != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(sm[w][r] - m);
        l += f * sl[w][r];
        o0 += f * so[w][r][d];
        o1 += f * so[w][r][d + 1];
      }
    }
    const float inv = l > 0.f ? __fdiv_rn(1.f, l) : (l == 0.f ? 0.f : l);
    const int row = row0 + r;
    __nv_bfloat16* out = a.O + (size_t(t0 + row / a.group) * a.heads * a.group + head * a.group +
                                row % a.group) * kDim + d;
    *reinterpret_cast<uint32_t*>(out) = bf16x2_bits(o0 * inv, o1 * inv);
  }
}

}  // namespace

cudaError_t launch_kv_attention(const LaunchCtx& c, const KvAttentionArgs& a) {
  const dim3 grid(ceil_div(a.max_q * a.group, kRows), a.heads, a.B);
  const bool e5 = a.fmt == FP8GEMM_FMT_E5M2;
  auto fn = a.dim == 128 ? (e5 ? kv_attention_kernel<128, true> : kv_attention_kernel<128, false>)
                         : (e5 ? kv_attention_kernel<64, true> : kv_attention_kernel<64, false>);
  fn<<<grid, 32 * kWarps, 0, c.stream>>>(a, c.status);
  return cudaGetLastError();
}

}  // namespace fp8gemm
