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
// Three launches: routing (one CTA), the up kernel (gate and up products,
// SwiGLU and quantisation) and the down kernel (down product and weighted sum).
//
// Bound by the chosen experts' weights, read once.  In both product kernels
// the K blocks of all output tiles of all chosen experts form one sequence
// that the CTAs share evenly, in runs, so every SM streams the same number of
// bytes whatever the number of experts.  A warp owns a share of a tile's rows
// and works on its own: one lane asks for the weights ahead (TMA into the
// warp's ring, across tile ends), and the 128-byte swizzle gives every lane its
// share of an m16n8k32 fragment without a bank conflict.  Weight rows are the
// 16-row side, tokens the 8-column side; a contraction's order is free, so a
// lane's share of a row's K block is 32 neighbouring bytes.  A tile that lies in
// several runs is joined from FP32 partials, in CTA order, by the CTA that
// finishes last: results do not depend on timing.
#include "common.cuh"
#include "f8_convert.cuh"
#include "moe_few.cuh"
#include "ptx.cuh"

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

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's share of one row's K block, bytes 32 t .. + 31.
struct Chunk {
  uint32_t w[8];
};

// Of an activation row, 0 past its K bytes (a multiple of 16).
__device__ __forceinline__ Chunk load_chunk(const uint8_t* row, int k0, int K, int t) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = k0 + 32 * t + 16 * i;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row != nullptr && k < K) v = *reinterpret_cast<const uint4*>(row + k);
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

// One K block of 16 weight rows (lo: rows 0-7, hi: rows 8-15) times 8 tokens.
__device__ __forceinline__ void mma_block(float (&d)[4], const Chunk& lo, const Chunk& hi,
                                          const Chunk& x) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    mma_e4m3(d, lo.w[2 * s], hi.w[2 * s], lo.w[2 * s + 1], hi.w[2 * s + 1], x.w[2 * s],
             x.w[2 * s + 1]);
}

// ------------------------------------------------------------------ routing
// Some (at most 8 NT) of the pairs that chose one expert: one pass over its weights.
struct Pass {
  int e, first, cnt, unused;  // pairs list[first .. first + cnt - 1]
};

// What routing leaves for the product kernels.  Pair p = token * k + choice.
struct Route {
  float* weight;  // [T k]
  int* list;      // [T k] pairs by expert, ascending within each
  Pass* pass;     // [T k]
  int* passes;    // how many
};

// A float as an unsigned number of the same order; NaN as -infinity.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (isnan(v)) v = -INFINITY;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);  // -0 and 0 tie
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One CTA: a warp per token chooses its experts; then a thread per expert
// counts and lists its pairs.
__global__ void __launch_bounds__(1024) moe_route_kernel(const float* __restrict__ logits, Route r,
                                                         int32_t* ids_out, float* w_out, int T,
                                                         int E, int k, int renormalise,
                                                         int per_pass) {
  constexpr int kPer = kMoeMaxExperts / 32;
  __shared__ __align__(16) int ids[kMoeMaxTokens * kMoeMaxTopK + 4];
  __shared__ int warp_pairs[32], warp_passes[32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  griddep_launch_dependents();
  griddep_wait();
  const int per = ceil_div(E, 32);  // values a lane holds
  for (int t = warp; t < T; t += 32) {
    float v[kPer];
    uint32_t key[kPer];
    uint32_t taken = 0;  // bit i: expert lane + 32 i is chosen already
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      v[i] = i < per && e < E ? logits[t * E + e] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      key[i] = order_key(v[i]);
      if (lane + 32 * i >= E) taken |= 1u << i;
    }
    float first = 0.f, sum = 0.f, mine = 0.f;
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0, at = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < per && !(taken >> i & 1) && (at == 0xffffffffu || key[i] > best)) {
          best = key[i];
          at = lane + 32 * i;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, at == 0xffffffffu ? 0u : best);
      at = __reduce_min_sync(0xffffffffu, best == top ? at : 0xffffffffu);
      float mine_v = -INFINITY;  // the chosen logit, from the lane that holds it
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == int(at / 32)) mine_v = v[i];
      float x = __shfl_sync(0xffffffffu, mine_v, at % 32);
      if (isnan(x)) x = -INFINITY;
      if (at % 32 == uint32_t(lane)) taken |= 1u << (at / 32);
      if (j == 0) first = x;
      const float p = x == -INFINITY ? 0.f : expf(x - first);
      sum += p;
      if (j == lane) {
        mine = p;
        ids_out[t * k + j] = int(at);
        ids[t * k + j] = int(at);
      }
    }
    if (!renormalise) {  // over all experts
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < per) sum += isnan(v[i]) || v[i] == -INFINITY ? 0.f : expf(v[i] - first);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < k) {
      const float w = sum > 0.f ? __fdiv_rn(mine, sum) : 0.f;
      w_out[t * k + lane] = w;
      r.weight[t * k + lane] = w;
    }
  }
  const int P = T * k;
  if (threadIdx.x < 4) ids[P + threadIdx.x] = -1;
  __syncthreads();
  const int e = threadIdx.x;  // E <= 512 of the 1024 threads
  int n = 0;
  if (e < E)
    for (int p = 0; p < P; p += 4) {
      const int4 q = *reinterpret_cast<const int4*>(ids + p);
      n += int(q.x == e) + int(q.y == e) + int(q.z == e) + int(q.w == e);
    }
  // exclusive sums over the experts of the pairs and of the passes
  const int m = ceil_div(n, per_pass);
  int before = n, pass = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, before, o), b = __shfl_up_sync(0xffffffffu, pass, o);
    if (lane >= o) {
      before += a;
      pass += b;
    }
  }
  if (lane == 31) {
    warp_pairs[warp] = before;
    warp_passes[warp] = pass;
  }
  __syncthreads();
  before -= n;
  pass -= m;
  for (int w = 0; w < warp; ++w) {
    before += warp_pairs[w];
    pass += warp_passes[w];
  }
  if (threadIdx.x == blockDim.x - 1) *r.passes = pass + m;
  if (n == 0) return;
  for (int i = 0; i < m; ++i)
    r.pass[pass + i] = Pass{e, before + i * per_pass, min(per_pass, n - i * per_pass), 0};
  for (int p = 0; p < P; ++p)
    if (ids[p] == e) r.list[before++] = p;
}

// ------------------------------------------------------------ product kernels
// A CTA's run of the unit sequence.
struct Run {
  long long U, per;
  long long u0, u1;
  __device__ Run(long long units) : U(units) {
    per = max((long long)kMinUnits, (U + gridDim.x - 1) / gridDim.x);
    u0 = blockIdx.x * per;
    u1 = min(U, u0 + per);
  }
};

// One warp's ring of weight tiles.
template <int kStages, int kStageBytes>
struct Ring {
  uint8_t* buf;
  uint64_t* bar;
  uint32_t phases = 0, in_flight = 0;  // bit s: parity to wait for; asked for

  __device__ uint8_t* stage(int s) const { return buf + s * kStageBytes; }
  // Waits for stage s; false if that ran out (or another warp's wait did).
  __device__ bool wait(int s, int* gave_up, int* never, int* status, unsigned long long limit_ns) {
    if (!mbar_wait(&bar[s], phases >> s & 1, gave_up, limit_ns)) {
      // results are void; what is still in flight lands first, or not at all
      *reinterpret_cast<volatile int*>(gave_up) = 1;
      raise_status(status, FP8GEMM_ERR_TIMEOUT);
      for (int k = 0; k < kStages; ++k)
        if (in_flight >> k & 1) mbar_wait(&bar[k], phases >> k & 1, never, limit_ns);
      return false;
    }
    phases ^= 1u << s;
    in_flight &= ~(1u << s);
    return true;
  }
};

struct Shared {
  uint64_t bars[kWarps][4];
  int gave_up, never, last_one;  // a wait ran out; always 0; this CTA joins
};

__device__ __forceinline__ uint8_t* init_shared(Shared& sh, uint8_t* raw, const CUtensorMap* map) {
  if (threadIdx.x == 0) {
    sh.gave_up = sh.never = 0;
    for (int i = 0; i < kWarps * 4; ++i) mbar_init(&sh.bars[0][i], 1);
    fence_mbar_init();
    tma_prefetch_desc(map);
  }
  __syncthreads();
  return raw + (1024u - (smem_addr(raw) & 1023u)) % 1024u;
}

// Gate and up products.  Unit: one K block of a tile (pass, 128 hidden
// columns); warp w takes hidden columns 32 w .. + 31 of it, rows of gate and of
// up alike, so that SwiGLU stays within a lane.
//   partial: [warp][fragment 0-3][n][element][lane] floats
template <int NT>
constexpr int kUpStages = NT == 4 ? 3 : 2;

template <int NT>
__global__ void __launch_bounds__(kThreads, kPerSm<NT>) moe_up_kernel(const MoeArgs a, const Route r,
                                                             const __grid_constant__ CUtensorMap map,
                                                             uint8_t* __restrict__ H8,
                                                             float* __restrict__ sH, int* counters,
                                                             float* parts, int* status) {
  constexpr int kPart = kWarps * 4 * NT * 4 * 32;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  __shared__ float amaxes[kWarps][8 * NT];
  __shared__ __align__(16) uint8_t codes[8 * NT][kBlockK];
  uint8_t* rings = init_shared(sh, raw, &map);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int Kb = ceil_div(a.H, kBlockK), Ib = ceil_div(a.I, kBlockK), Rb = ceil_div(2 * a.I, kBlockK);
  Ring<kUpStages<NT>, 64 * kBlockK> ring{rings + warp * kUpStages<NT> * 64 * kBlockK, sh.bars[warp]};
  griddep_wait();
  griddep_launch_dependents();  // all before this kernel is complete: the next may read weights
  const Run run((long long)*r.passes * Ib * Kb);
  if (run.u0 >= run.u1) return;

  // the unit that is asked for next, kUpStages ahead of the one in use
  long long ask = run.u0;
  int ask_tile = int(ask / Kb), ask_kb = int(ask % Kb), ask_stage = 0;
  int ask_e = r.pass[ask_tile / Ib].e;
  auto fetch = [&]() {
    if (ask >= run.u1) return;
    ring.in_flight |= 1u << ask_stage;
    if (lane == 0) {
      const int row = ask_e * 2 * a.I + ask_tile % Ib * kBlockK + 32 * warp;
      uint8_t* s = ring.stage(ask_stage);
      mbar_arrive_expect_tx(&ring.bar[ask_stage], 64 * kBlockK);
      tma_load_2d(s, &map, &ring.bar[ask_stage], ask_kb * kBlockK, row);
      tma_load_2d(s + 32 * kBlockK, &map, &ring.bar[ask_stage], ask_kb * kBlockK, row + a.I);
    }
    ask_stage = ask_stage + 1 == kUpStages<NT> ? 0 : ask_stage + 1;
    ++ask;
    if (++ask_kb == Kb) {
      ask_kb = 0;
      ++ask_tile;
      if (ask < run.u1 && ask_tile % Ib == 0) ask_e = r.pass[ask_tile / Ib].e;
    }
  };
#pragma unroll
  for (int i = 0; i < kUpStages<NT>; ++i) fetch();

  // what a unit needs besides weights, loaded a unit ahead
  struct Side {
    Chunk x[NT];
    float sx[NT][2], sg, su[2];
  } next;
  Pass pass = {};
  int side_tile = -1;
  int tok[NT], col[NT][2];  // the token this lane loads; those of its two columns (-1: none)
  const float *sg = nullptr, *su[2] = {};
  auto side = [&](long long u) {
    const int tile = int(u / Kb), kb = int(u - (long long)tile * Kb);
    if (tile != side_tile) {
      if (side_tile < 0 || tile / Ib != side_tile / Ib) {
        pass = r.pass[tile / Ib];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          tok[n] = 8 * n + g < pass.cnt ? r.list[pass.first + 8 * n + g] / a.k : -1;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            col[n][c] = 8 * n + 2 * t + c < pass.cnt ? r.list[pass.first + 8 * n + 2 * t + c] / a.k : -1;
        }
      }
      side_tile = tile;
      const int i0 = tile % Ib * kBlockK;
      const float* s = a.s1 + size_t(pass.e) * Rb * Kb;
      sg = s + size_t(i0 / kBlockK) * Kb;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        su[m] = s + size_t(min((a.I + i0 + 32 * warp + 16 * m) / kBlockK, Rb - 1)) * Kb;
    }
    next.sg = sg[kb];
    next.su[0] = su[0][kb];
    next.su[1] = su[1][kb];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= pass.cnt) break;
      next.x[n] = load_chunk(tok[n] >= 0 ? a.A + size_t(tok[n]) * a.H : nullptr, kb * kBlockK, a.H, t);
#pragma unroll
      for (int c = 0; c < 2; ++c) next.sx[n][c] = col[n][c] >= 0 ? a.sA[size_t(col[n][c]) * Kb + kb] : 0.f;
    }
  };
  side(run.u0);

  float acc[4][NT][4] = {};
  int stage = 0;
  bool dead = false;
  for (long long u = run.u0; u < run.u1; ++u) {
    const Side here = next;
    const Pass at = pass;
    const int tile = side_tile;
    if (u + 1 < run.u1) side(u + 1);
    // After a wait that ran out the warp only keeps the others' barriers company.
    dead = dead || !ring.wait(stage, &sh.gave_up, &sh.never, status, a.wait_ns);
    const uint8_t* w = ring.stage(stage);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const Chunk lo = tile_chunk(w, 16 * m + g, t), hi = tile_chunk(w, 16 * m + 8 + g, t);
      const float sw = m < 2 ? here.sg : here.su[m - 2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
        float d[4] = {};
        mma_block(d, lo, hi, here.x[n]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = fmaf(d[c], here.sx[n][c & 1] * sw, acc[m][n][c]);
      }
    }
    __syncwarp();  // the stage has been read
    if (!dead) fetch();
    stage = stage + 1 == kUpStages<NT> ? 0 : stage + 1;
    const long long tile0 = (long long)tile * Kb;
    if (u + 1 < run.u1 && u + 1 < tile0 + Kb) continue;

    // the run's share of this tile is done
    const bool whole = tile0 >= run.u0 && tile0 + Kb <= run.u1;
    const int first = int(tile0 / run.per), last = int((tile0 + Kb - 1) / run.per);
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
      const int i0 = tile % Ib * kBlockK;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= at.cnt) break;
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float gate = acc[m][n][c];
            float h = __fdiv_rn(gate, 1.f + expf(-gate)) * acc[2 + m][n][c];
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
            sH[size_t(r.list[at.first + j]) * Ib + tile % Ib] = s;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              codes[j][32 * warp + 16 * m + 8 * e + g] =
                  top != 0.f ? uint8_t(cvt_f8x2<false>(__fdiv_rn(acc[m][n][2 * e + c], s), 0.f)) : 0;
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
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.f;
  }
}

// Down product and weighted sum.  Unit: one K block of one pass for a tile of
// 128 output columns; warp w takes columns 32 w .. + 31 and keeps a sum per token
// in shared memory that no other warp touches.
//   partial: [warp][token][32] floats
constexpr int kDownStages = 4;
constexpr int kSumRow = 36;  // floats from token to token: lanes of a fragment hit all banks

template <int NT>
__global__ void __launch_bounds__(kThreads, kPerSm<NT>) moe_down_kernel(const MoeArgs a, const Route r,
                                                               const __grid_constant__ CUtensorMap map,
                                                               const uint8_t* H8, const float* sH,
                                                               int* counters, float* parts,
                                                               int* status) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  uint8_t* rings = init_shared(sh, raw, &map);
  float* all_sums = reinterpret_cast<float*>(rings + kWarps * kDownStages * 32 * kBlockK);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int Kb = ceil_div(a.I, kBlockK), Hb = ceil_div(a.H, kBlockK);
  float* sums = all_sums + warp * a.T * kSumRow;
  for (int i = lane; i < a.T * kSumRow; i += 32) sums[i] = 0.f;
  Ring<kDownStages, 32 * kBlockK> ring{rings + warp * kDownStages * 32 * kBlockK, sh.bars[warp]};
  // The up kernel let this one start after everything before it was complete:
  // routing and weights may be read, the hidden activations not yet.
  const int passes = __ldcg(r.passes);
  const long long per_tile = (long long)passes * Kb;
  const Run run(Hb * per_tile);
  if (run.u0 >= run.u1) {
    griddep_wait();
    return;
  }
  long long ask = run.u0;
  int ask_tile = int(ask / per_tile), ask_stage = 0;
  int ask_pass = int((ask - ask_tile * per_tile) / Kb), ask_kb = int(ask % Kb);
  int ask_e = __ldcg(&r.pass[ask_pass].e);
  auto fetch = [&]() {
    if (ask >= run.u1) return;
    ring.in_flight |= 1u << ask_stage;
    if (lane == 0) {
      mbar_arrive_expect_tx(&ring.bar[ask_stage], 32 * kBlockK);
      tma_load_2d(ring.stage(ask_stage), &map, &ring.bar[ask_stage], ask_kb * kBlockK,
                  ask_e * a.H + ask_tile * kBlockK + 32 * warp);
    }
    ask_stage = (ask_stage + 1) % kDownStages;
    ++ask;
    if (++ask_kb == Kb) {
      ask_kb = 0;
      if (++ask_pass == passes) {
        ask_pass = 0;
        ++ask_tile;
      }
      if (ask < run.u1) ask_e = __ldcg(&r.pass[ask_pass].e);
    }
  };
#pragma unroll
  for (int i = 0; i < kDownStages; ++i) fetch();
  griddep_launch_dependents();
  griddep_wait();

  struct Side {
    Chunk x[NT];
    float sx[NT][2], sw;
  } next;
  Pass pass = {};
  int tile = int(run.u0 / per_tile), pi = int((run.u0 - tile * per_tile) / Kb), kb = int(run.u0 % Kb);
  int row[NT], col[NT][2];  // the pair this lane loads; those of its two columns (-1: none)
  const float* sw = nullptr;
  auto enter = [&]() {  // the side loads enter pass pi of a tile
    pass = r.pass[pi];
    sw = a.s2 + (size_t(pass.e) * Hb + tile) * Kb;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      row[n] = 8 * n + g < pass.cnt ? r.list[pass.first + 8 * n + g] : -1;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        col[n][c] = 8 * n + 2 * t + c < pass.cnt ? r.list[pass.first + 8 * n + 2 * t + c] : -1;
    }
  };
  auto side = [&]() {
    next.sw = sw[kb];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (8 * n >= pass.cnt) break;
      next.x[n] = load_chunk(row[n] >= 0 ? H8 + size_t(row[n]) * a.I : nullptr, kb * kBlockK, a.I, t);
#pragma unroll
      for (int c = 0; c < 2; ++c) next.sx[n][c] = col[n][c] >= 0 ? sH[size_t(col[n][c]) * Kb + kb] : 0.f;
    }
  };
  enter();
  side();

  float acc[2][NT][4] = {};
  int stage = 0;
  bool dead = false;
  for (long long u = run.u0; u < run.u1; ++u) {
    const Side here = next;
    const int cnt = pass.cnt, this_tile = tile;
    int here_col[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      here_col[n][0] = col[n][0];
      here_col[n][1] = col[n][1];
    }
    const bool pass_ends = kb + 1 == Kb || u + 1 == run.u1;
    if (u + 1 < run.u1) {
      if (++kb == Kb) {
        kb = 0;
        if (++pi == passes) {
          pi = 0;
          ++tile;
        }
        enter();
      }
      side();
    }
    // After a wait that ran out the warp only keeps the others' barriers company.
    dead = dead || !ring.wait(stage, &sh.gave_up, &sh.never, status, a.wait_ns);
    const uint8_t* w = ring.stage(stage);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const Chunk lo = tile_chunk(w, 16 * m + g, t), hi = tile_chunk(w, 16 * m + 8 + g, t);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n >= cnt) break;
        float d[4] = {};
        mma_block(d, lo, hi, here.x[n]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = fmaf(d[c], here.sx[n][c & 1] * here.sw, acc[m][n][c]);
      }
    }
    __syncwarp();  // the stage has been read
    if (!dead) fetch();
    stage = (stage + 1) % kDownStages;
    if (!pass_ends) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (here_col[n][c] >= 0) {
          const float wt = r.weight[here_col[n][c]];
          float* s = sums + here_col[n][c] / a.k * kSumRow + g;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              s[16 * m + 8 * e] = fmaf(acc[m][n][2 * e + c], wt, s[16 * m + 8 * e]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) acc[m][n][c] = acc[m][n][2 + c] = 0.f;
      }
    __syncwarp();
    const long long tile0 = this_tile * per_tile;
    if (u + 1 < run.u1 && u + 1 < tile0 + per_tile) continue;

    // the run's share of this tile is done
    const bool whole = tile0 >= run.u0 && tile0 + per_tile <= run.u1;
    const int first = int(tile0 / run.per), last = int((tile0 + per_tile - 1) / run.per);
    const size_t part_size = size_t(kWarps) * a.T * 32;
    const int h0 = this_tile * kBlockK + 32 * warp;
    if (!whole) {
      float* part = parts + (2 * blockIdx.x + (tile0 >= run.u0 ? 1 : 0)) * part_size + warp * a.T * 32;
      for (int i = lane; i < a.T * 8; i += 32)
        reinterpret_cast<float4*>(part)[i] =
            *reinterpret_cast<const float4*>(sums + i / 8 * kSumRow + i % 8 * 4);
      __syncthreads();
      if (threadIdx.x == 0) {
        sh.last_one = atomic_add_acq_rel_gpu(counters + first, 1) == last - first;
        if (sh.last_one) counters[first] = 0;
      }
      __syncthreads();
      if (sh.last_one)
        for (int i = lane; i < a.T * 8; i += 32) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int q = first; q <= last; ++q) {
            const float4 p = __ldcg(reinterpret_cast<const float4*>(
                                        parts + (2 * q + (q == first ? 1 : 0)) * part_size + warp * a.T * 32) + i);
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
          }
          *reinterpret_cast<float4*>(sums + i / 8 * kSumRow + i % 8 * 4) = v;
        }
      __syncwarp();
    }
    if (whole || sh.last_one)
      for (int i = lane; i < a.T * 8; i += 32) {
        const int h = h0 + i % 8 * 4;
        if (h >= a.H) continue;  // H is a multiple of 16
        const float* s = sums + i / 8 * kSumRow + i % 8 * 4;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s[0], s[1]), hi = __floats2bfloat162_rn(s[2], s[3]);
        uint2 o;
        o.x = *reinterpret_cast<const uint32_t*>(&lo);
        o.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(a.D + size_t(i / 8) * a.H + h) = o;
      }
    __syncthreads();  // last_one is free
    for (int i = lane; i < a.T * kSumRow; i += 32) sums[i] = 0.f;
    __syncwarp();
  }
}

// ------------------------------------------------------------------- launches
int fragments(const MoeArgs& a) { return a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4; }

struct Layout {
  size_t counters, h8, sh, weight, list, pass, passes, up, down, total;
};

Layout layout(const LaunchCtx& c, const MoeArgs& a) {
  const size_t P = size_t(a.T) * a.k, grid = size_t(kMaxPerSm) * c.num_sms;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  Layout l;
  l.counters = take(2 * grid * 4);  // first: its place does not depend on the call's sizes
  l.h8 = take(P * a.I);
  l.sh = take(P * ceil_div(a.I, kBlockK) * 4);
  l.weight = take(P * 4);
  l.list = take(P * 4);
  l.pass = take(P * sizeof(Pass));
  l.passes = take(4);
  l.up = take(2 * grid * kWarps * 4 * fragments(a) * 4 * 32 * 4);
  l.down = take(2 * grid * kWarps * a.T * 32 * 4);
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
  const int grid = kPerSm<NT> * c.num_sms;
  const size_t up_smem = 1024 + size_t(kWarps) * kUpStages<NT> * 64 * kBlockK;
  const size_t down_smem =
      1024 + size_t(kWarps) * (kDownStages * 32 * kBlockK + size_t(a.T) * kSumRow * 4);
  const size_t down_most =
      1024 + size_t(kWarps) * (kDownStages * 32 * kBlockK + size_t(kMoeMaxTokens) * kSumRow * 4);
  auto up = moe_up_kernel<NT>;
  auto down = moe_down_kernel<NT>;
  static SmemLimit up_limit, down_limit;
  if (cudaError_t e = up_limit.raise(reinterpret_cast<const void*>(up), up_smem)) return e;
  if (cudaError_t e = down_limit.raise(reinterpret_cast<const void*>(down), down_most)) return e;
  if (cudaError_t e = launch_dependent(c, moe_route_kernel, 1, 1024, 0, a.logits, r, a.ids,
                                       a.weights, a.T, a.E, a.k, a.renormalise, 8 * NT))
    return e;
  if (cudaError_t e = launch_dependent(c, up, grid, kThreads, up_smem, a, r, m1, H8, sH, counters,
                                       reinterpret_cast<float*>(ws + l.up), c.status))
    return e;
  return launch_dependent(c, down, grid, kThreads, down_smem, a, r, m2, H8, sH,
                          counters + kMaxPerSm * c.num_sms, reinterpret_cast<float*>(ws + l.down), c.status);
}

}  // namespace

size_t moe_few_workspace_bytes(const LaunchCtx& c, const MoeArgs& a) { return layout(c, a).total; }

cudaError_t launch_moe_few(const LaunchCtx& c, const MoeArgs& a, void* workspace, int* launches) {
  char* ws = static_cast<char*>(workspace);
  const Layout l = layout(c, a);
  const Route r{reinterpret_cast<float*>(ws + l.weight), reinterpret_cast<int*>(ws + l.list),
                reinterpret_cast<Pass*>(ws + l.pass), reinterpret_cast<int*>(ws + l.passes)};
  *launches = 3;
  switch (fragments(a)) {
    case 1: return launch_nt<1>(c, a, r, ws, l);
    case 2: return launch_nt<2>(c, a, r, ws, l);
    default: return launch_nt<4>(c, a, r, ws, l);
  }
}

}  // namespace fp8gemm
