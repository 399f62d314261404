// gemm_gated.cu -- the gated feed-forward block's FP8 products with what follows them in one
// kernel, and its gradient.
//
// Forward   u = A W1^T (gate rows, then up rows; block scales as in gemm_tc.cu)
//           h = silu(u_gate) u_up,  one scale and FP8 codes per 1x128 block of h
// Backward  dh = dY W2 (as dY W2T^T),  s = 1 / (1 + e^-g) of the kept gate g and up u:
//           dg = dh u s (1 + g (1 - s)),  du = dh g s,  codes of both per 1x128 block
//
// The products are those of gemm_tc.cu -- operands by TMA into a ring, one tcgen05
// contraction per 128-wide K block into one of two TMEM buffers, each block's partial
// promoted with its scale product into FP32 registers -- and the same CTA layout (384
// threads; see there).  What differs is which columns meet in a thread:
//   forward   a tile is 128 rows of 128 columns of h: its 256 accumulator columns are
//             gate 0-63, up 0-63, gate 64-127, up 64-127 (four boxes of W1's rows a K
//             block), so that each promotion thread holds 64 gate values and the up values
//             of the same columns, and a row's maximum is one exchange between two threads
//   backward  256 columns of dh: each promotion thread holds one whole 1x128 block of a row
// so the activations never leave the chip in 16 or 32 bits.  The backward form's gate and up values come
// through the operand ring too, behind the tile's last K block (direct loads of 16 bytes a row, each
// from another line, took longer than the product: 257 us at 8192 x 2048 x 7168); du waits in their places
// until the block's maximum is known, and the 16-bit gradients leave from there.  (Four promotion
// warpgroups of 64 columns each, to hide the TMEM loads' latency and shorten the epilogue, were slower:
// 178 us forward at 4096 x 2048 x 7168 for 124.)
//
// Bound by the tensor cores and the promotion for prompts: 4096 x 7168 to 2 x 2048 columns take 118 us where
// the plain product of that size takes 106 (four waves, the last one of 56 tiles: splitting that one along K as
// a launch of its own won 1 us here and lost 9 in the gradient), the gradient of 8192 rows 149 us where
// the product takes 107; its epilogue is 10 us a tile.  By latency and the weights' bytes for a few tokens
// (29 MB in 10.8 us): then all tiles fit in one wave, and each is split along K over a cluster (as in
// gemm_tc.cu), whose CTAs share the rows of the epilogue.
#include <cstring>

#include "common.cuh"
#include "f8_convert.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8gemm {
namespace {

constexpr int kGroupM = 16;  // M blocks per rasterisation group
constexpr int kBN = 256;     // accumulator columns of a tile
constexpr int kStages = 4;
constexpr int kGroups = 2;            // promotion warpgroups
constexpr int kCols = kBN / kGroups;  // accumulator columns of a thread
constexpr int kPromoWarps = 4 * kGroups;
constexpr int kTmaWarp = kPromoWarps, kMmaWarp = kPromoWarps + 1;
constexpr int kThreads = 128 * (kGroups + 1);
// 65536 / 384 -> 168 registers at launch; 128 * 72 + 256 * 216 = 384 * 168
constexpr uint32_t kLowRegs = 72, kHighRegs = 216;
static_assert(kGroups * kHighRegs + kLowRegs <= 3 * 168, "register split");
constexpr int kABytes = kBlockM * kBlockK, kBBytes = kBN * kBlockK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kPitch = kBN + 4;  // floats of a staged row (split tiles)
constexpr int kBoxBytes = kBlockM * 128;  // 64 columns of gate or up values: one of three in a stage
constexpr int kGuStages = 3;              // stages that a tile's eight boxes take
constexpr size_t kSmemBytes = 1024 + size_t(kStages) * kStageBytes + 2 * kGroups * kBlockM * 4 + 512;
static_assert(kSmemBytes <= 232448, "227 KB of shared memory per CTA");
static_assert(size_t(kBlockM) * kPitch * 4 <= size_t(kStages) * kStageBytes, "staging fits the ring");

// Columns of h (or dh) of a tile.
template <bool kGrad>
__host__ __device__ constexpr int tile_cols() {
  return kGrad ? kBN : kBN / 2;
}

struct GatedTile {
  int row0, rows, col0;  // first row, rows that exist, first column of h
};

template <bool kGrad>
__device__ __forceinline__ GatedTile gated_tile(const GatedArgs& a, int t) {
  const int num_n = ceil_div(a.I, tile_cols<kGrad>()), num_m = ceil_div(a.M, kBlockM);
  const int per_group = kGroupM * num_n;
  const int first_m = t / per_group * kGroupM, gs = min(kGroupM, num_m - first_m);
  const int r = t % per_group;
  GatedTile w;
  w.row0 = (first_m + r % gs) * kBlockM;
  w.rows = min(kBlockM, a.M - w.row0);
  w.col0 = r / gs * tile_cols<kGrad>();
  return w;
}

// e^-x, to FP32's rounding (relative error 2^-22 and x's own).
__device__ __forceinline__ float exp_minus(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * -1.4426950408889634f));
  return r;
}

// 1 / (1 + e^-g), to a few units in FP32's last place; 0 where it is below FP32's normal numbers (g below -87.3).
__device__ __forceinline__ float sigmoid(float g) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp_minus(g)));
  return r;
}

__device__ __forceinline__ float swiglu(float g, float u) { return g * sigmoid(g) * u; }

// dg and du of one element.  In this order: s (1 + g (1 - s)) is 1.1 at most, so that what leaves FP32 on the way (u g
// where s is 0) is no part of it.
__device__ __forceinline__ float2 swiglu_grad(float dh, float g, float u) {
  const float s = sigmoid(g), ds = dh * s;
  return make_float2(ds * fmaf(g, 1.f - s, 1.f) * u, ds * g);
}

// Sixteen values to codes of one scale, stored at p.
__device__ __forceinline__ void store_codes16(uint8_t* p, const float (&v)[16], const Reciprocal& s, bool e5m2) {
  uint32_t c[4];
  if (s.safe) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = quotient(v[4 * i], s), b = quotient(v[4 * i + 1], s), x = quotient(v[4 * i + 2], s),
                  y = quotient(v[4 * i + 3], s);
      c[i] = e5m2 ? cvt_f8x2<true>(a, b) | (cvt_f8x2<true>(x, y) << 16) : cvt_f8x2<false>(a, b) | (cvt_f8x2<false>(x, y) << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      c[i] = s.s == 0.f ? 0u : e5m2 ? quant4<true>(x, s.s) : quant4<false>(x, s.s);
    }
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(c[0], c[1], c[2], c[3]);
}

template <bool kE5M2>
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], const Reciprocal& s) {
  const float4 x = make_float4(v[0], v[1], v[2], v[3]);
  if (s.safe) return quant4<kE5M2>(x, s);
  return s.s == 0.f ? 0u : quant4<kE5M2>(x, s.s);
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---- split tiles: a warp's row of one 1x128 block, four columns a lane
template <bool kE5M2>
__device__ __forceinline__ void finish_h(const GatedArgs& a, int row, int col, int lane, float4 g,
                                         float4 u) {
  const bool in = col + 4 * lane < a.I;
  float h[4] = {swiglu(g.x, u.x), swiglu(g.y, u.y), swiglu(g.z, u.z), swiglu(g.w, u.w)};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max_nan(top, in ? fabsf(h[i]) : 0.f);
  const Reciprocal s = reciprocal(block_scale<kE5M2>(warp_max_nan(top)));
  if (lane == 0) a.sQ[size_t(row) * ceil_div(a.I, kBlockK) + col / kBlockK] = s.s;
  if (!in) return;
  *reinterpret_cast<uint32_t*>(a.Q + size_t(row) * a.I + col + 4 * lane) = codes4<kE5M2>(h, s);
  if (a.GU) {
    __nv_bfloat16* o = a.GU + size_t(row) * 2 * a.I + col + 4 * lane;
    *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2_bits(g.x, g.y), bf16x2_bits(g.z, g.w));
    *reinterpret_cast<uint2*>(o + a.I) = make_uint2(bf16x2_bits(u.x, u.y), bf16x2_bits(u.z, u.w));
  }
}

template <bool kE5M2>
__device__ __forceinline__ void finish_dgu(const GatedArgs& a, int row, int col, int lane, float4 dh4) {
  const int Ip = ceil_div(a.I, kBlockK) * kBlockK;
  const bool in = col + 4 * lane < a.I;
  float dg[4] = {}, du[4] = {};
  if (in) {
    const __nv_bfloat16* p = a.GU + size_t(row) * 2 * a.I + col + 4 * lane;
    const uint2 g = *reinterpret_cast<const uint2*>(p), u = *reinterpret_cast<const uint2*>(p + a.I);
    const uint32_t gw[2] = {g.x, g.y}, uw[2] = {u.x, u.y};
    const float dh[4] = {dh4.x, dh4.y, dh4.z, dh4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gv = __uint_as_float(i % 2 ? gw[i / 2] & 0xffff0000u : gw[i / 2] << 16);
      const float uv = __uint_as_float(i % 2 ? uw[i / 2] & 0xffff0000u : uw[i / 2] << 16);
      const float2 d = swiglu_grad(dh[i], gv, uv);
      dg[i] = d.x;
      du[i] = d.y;
    }
  }
  float top_g = 0.f, top_u = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top_g = max_nan(top_g, fabsf(dg[i]));
    top_u = max_nan(top_u, fabsf(du[i]));
  }
  const Reciprocal sg = reciprocal(block_scale<kE5M2>(warp_max_nan(top_g)));
  const Reciprocal su = reciprocal(block_scale<kE5M2>(warp_max_nan(top_u)));
  if (lane == 0) {
    float* sq = a.sQ + size_t(row) * (2 * Ip / kBlockK) + col / kBlockK;
    sq[0] = sg.s;
    sq[Ip / kBlockK] = su.s;
  }
  uint8_t* q = a.Q + size_t(row) * 2 * Ip + col + 4 * lane;
  *reinterpret_cast<uint32_t*>(q) = in ? codes4<kE5M2>(dg, sg) : 0u;
  *reinterpret_cast<uint32_t*>(q + Ip) = in ? codes4<kE5M2>(du, su) : 0u;
  if (in && a.dGU) {
    __nv_bfloat16* o = a.dGU + size_t(row) * 2 * a.I + col + 4 * lane;
    *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2_bits(dg[0], dg[1]), bf16x2_bits(dg[2], dg[3]));
    *reinterpret_cast<uint2*>(o + a.I) = make_uint2(bf16x2_bits(du[0], du[1]), bf16x2_bits(du[2], du[3]));
  }
}

// kSplit: cluster c of args.split CTAs computes tile c, CTA rank r the r-th share of its K blocks.
// tmG, tmU: gate and up values, and tmDG, tmDU their gradients (backward, whole tiles).
template <bool kGrad, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_gated_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
                      const __grid_constant__ CUtensorMap tmDG, const __grid_constant__ CUtensorMap tmDU,
                      const __grid_constant__ GatedArgs args, int* status) {
  constexpr bool kRingGu = kGrad && !kSplit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + kStages * kABytes;
  float* tops = reinterpret_cast<float*>(smem + kStages * kStageBytes);  // [2][kGroups][kBlockM]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(tops + 2 * kGroups * kBlockM);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* tfull_bar = empty_bar + kStages;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* row_bar = tempty_bar + 2;  // the promotion warps of the same rows
  uint64_t* gu_bar = row_bar + 4;      // a tile's gate and up values have been used
  uint64_t* drain_bar = gu_bar + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], kPromoWarps);
    }
    for (int p = 0; p < 4; ++p) mbar_init(&row_bar[p], kGroups);
    mbar_init(gu_bar, kPromoWarps);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, 2 * kBN);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if constexpr (kRingGu) {
      tma_prefetch_desc(&tmG);
      tma_prefetch_desc(&tmU);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // a programmatic dependent: nothing below may read before the stream's earlier work is complete
  griddep_wait();
  griddep_launch_dependents();

  const int Kb = ceil_div(args.K, kBlockK);
  const int total = ceil_div(args.M, kBlockM) * ceil_div(args.I, tile_cols<kGrad>());
  int t_begin = blockIdx.x, t_step = gridDim.x, kb0 = 0, kb1 = Kb, part = 0;
  if constexpr (kSplit) {
    part = int(cluster_ctarank());
    t_begin = blockIdx.x / args.split;
    t_step = total;  // one tile
    kb0 = part * Kb / args.split;
    kb1 = (part + 1) * Kb / args.split;
  }
  auto fail = [&]() {
    *abort_flag = 1;
    raise_status(status, FP8GEMM_ERR_TIMEOUT);
  };
  // A whole warp's wait, with one outcome: the TMEM loads behind it are the warp's.
  auto warp_wait = [&](uint64_t* b, uint32_t parity) {
    uint64_t t0 = 0;
    while (!__all_sync(0xffffffffu, mbar_try_wait(b, parity))) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, *abort_flag != 0 || now - t0 > args.wait_ns)) return false;
    }
    return true;
  };

  if (warp == kTmaWarp) {
    regs_decrease<kLowRegs>();
    if (lane == 0) {
      uint32_t it = 0;          // uses of the ring
      uint32_t was_gu = 0;      // bit s: stage s held gate and up values last
      uint32_t parity = 0xf;    // bit s: of the next completion of empty_bar[s] to wait for
      uint32_t gu_tiles = 0;
      // the stage's last contents have been used
      auto free_stage = [&](int s) {
        bool ok;
        if (kRingGu && (was_gu >> s & 1u)) {
          ok = mbar_wait(gu_bar, (gu_tiles - 1) & 1, abort_flag, args.wait_ns);
        } else {
          ok = mbar_wait(&empty_bar[s], parity >> s & 1u, abort_flag, args.wait_ns);
          parity ^= 1u << s;
        }
        if (!ok) fail();
        return ok;
      };
      bool ok = true;
      for (int t = t_begin; t < total && ok; t += t_step) {
        const GatedTile w = gated_tile<kGrad>(args, t);
        if constexpr (kRingGu)  // what the epilogue will read, into the L2 meanwhile
          for (int h = 0; h < 4; ++h) {
            tma_prefetch_l2_2d(&tmG, w.col0 + 64 * h, w.row0);
            tma_prefetch_l2_2d(&tmU, w.col0 + 64 * h, w.row0);
          }
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (!(ok = free_stage(s))) break;
          was_gu &= ~(1u << s);
          mbar_arrive_expect_tx(&full_bar[s], kStageBytes);
          tma_load_2d(smA + s * kABytes, &tmA, &full_bar[s], kb * kBlockK, w.row0);
          uint8_t* b = smB + s * kBBytes;
          if constexpr (kGrad) {
            tma_load_2d(b, &tmB, &full_bar[s], kb * kBlockK, w.col0);
          } else {
#pragma unroll 1
            for (int i = 0; i < 4; ++i)
              tma_load_2d(b + i * (kBBytes / 4), &tmB, &full_bar[s], kb * kBlockK,
                          w.col0 + 64 * (i / 2) + (i % 2 ? args.I : 0));
          }
        }
        if constexpr (kRingGu) {
#pragma unroll 1
          for (int g = 0; g < kGuStages && ok; ++g, ++it) {
            const int s = it % kStages, boxes = g < 2 ? 3 : 2;
            if (!(ok = free_stage(s))) break;
            was_gu |= 1u << s;
            mbar_arrive_expect_tx(&full_bar[s], boxes * kBoxBytes);
            for (int i = 0; i < boxes; ++i) {  // box 2 h: gate values of columns 64 h .. 64 h + 63, 2 h + 1: up values
              const int box = 3 * g + i;
              tma_load_2d(i == 0 ? smA + s * kABytes : smB + s * kBBytes + (i - 1) * kBoxBytes,
                          box % 2 ? &tmU : &tmG, &full_bar[s], w.col0 + 64 * (box / 2), w.row0);
            }
          }
          ++gu_tiles;
        }
      }
      // let the last copies into each stage land before the CTA can exit
      const uint32_t n = it < uint32_t(kStages) ? it : uint32_t(kStages);
      for (uint32_t i = it - n; i < it; ++i) mbar_drain(&full_bar[i % kStages], (i / kStages) & 1);
    }
  } else if (warp == kMmaWarp) {
    regs_decrease<kLowRegs>();
    if (lane == 0) {
      const uint32_t idesc = idesc_f8_f32(kBlockM, kBN, uint32_t(args.a_fmt), uint32_t(args.b_fmt));
      const uint64_t a_desc = smem_desc_sw128_kmajor(smem_addr(smA)), b_desc = smem_desc_sw128_kmajor(smem_addr(smB));
      uint32_t it = 0, n_mma = 0;
      bool ok = true;
      for (int t = t_begin; t < total && ok; t += t_step) {
        for (int kb = kb0; kb < kb1; ++kb, ++it, ++n_mma) {
          const int s = it % kStages, buf = n_mma & 1;
          if (!mbar_wait(&tempty_bar[buf], ((n_mma / 2) & 1) ^ 1, abort_flag, args.wait_ns) ||
              !mbar_wait(&full_bar[s], (it / kStages) & 1, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kBlockK / 32; ++k)
            umma_e4m3(tmem_base + buf * kBN, a_desc + ((s * kABytes + k * 32) >> 4), b_desc + ((s * kBBytes + k * 32) >> 4),
                      idesc, k > 0 ? 1u : 0u);
          umma_commit(&empty_bar[s]);
          umma_commit(&tfull_bar[buf]);
        }
        if constexpr (kRingGu) {
          // Each use of a stage is seen in turn, these too: a wait for a barrier's next phase but one would end
          // at once.
          for (int g = 0; g < kGuStages && ok; ++g, ++it)
            if (!mbar_wait(&full_bar[it % kStages], (it / kStages) & 1, abort_flag, args.wait_ns)) {
              fail();
              ok = false;
            }
        }
      }
      if (n_mma > 0) {  // every issued MMA has finished before TMEM is released
        umma_commit(drain_bar);
        mbar_drain(drain_bar, 0);
      }
    }
  } else if (warp < kPromoWarps) {
    regs_increase<kHighRegs>();
    const int wg = warp / 4;
    const int row = (warp % 4) * 32 + lane;  // TMEM lane = tile row
    const uint32_t taddr0 = tmem_base + (uint32_t((warp % 4) * 32) << 16) + wg * kCols;
    const int Nb = ceil_div(kGrad ? args.I : 2 * args.I, kBlockK);
    uint32_t n_mma = 0, it = 0, tiles = 0;
    bool ok = true;
    for (int t = t_begin; t < total && ok; t += t_step, ++tiles) {
      const GatedTile w = gated_tile<kGrad>(args, t);
      const bool row_ok = row < w.rows;
      const int col = w.col0 + wg * (tile_cols<kGrad>() / kGroups);  // the thread's first column of h
      // The up rows of W1 may begin inside a 128-row scale block: of the thread's 64 up columns the first
      // 16 n_low belong to one block, the rest to the next.
      const int b0 = min(col / kBlockK, Nb - 1);
      const int b1 = kGrad ? b0 : min((args.I + col) / kBlockK, Nb - 1);
      const int b2 = kGrad ? b0 : min(b1 + 1, Nb - 1);
      const int n_low = kGrad ? 4 : (kBlockK - (args.I + col) % kBlockK) / 16;
      const float* sa_ptr = args.sA + size_t(w.row0 + (row_ok ? row : 0)) * Kb;
      const float* s0_ptr = args.sB + size_t(b0) * Kb;
      const float* s1_ptr = args.sB + size_t(b1) * Kb;
      const float* s2_ptr = args.sB + size_t(b2) * Kb;
      float2 acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      float sa = __ldg(sa_ptr + kb0), s0 = __ldg(s0_ptr + kb0);
      float s1 = kGrad ? s0 : __ldg(s1_ptr + kb0), s2 = kGrad ? s0 : __ldg(s2_ptr + kb0);
      for (int kb = kb0; kb < kb1; ++kb, ++n_mma) {
        const float c0 = sa * s0, c1 = kGrad ? c0 : sa * s1, c2 = kGrad ? c0 : sa * s2;
        if (kb + 1 < kb1) {
          sa = __ldg(sa_ptr + kb + 1);
          s0 = __ldg(s0_ptr + kb + 1);
          if constexpr (!kGrad) {
            s1 = __ldg(s1_ptr + kb + 1);
            s2 = __ldg(s2_ptr + kb + 1);
          }
        }
        const int buf = n_mma & 1;
        if (!__all_sync(0xffffffffu, mbar_try_wait(&tfull_bar[buf], (n_mma / 2) & 1)) &&  // (most find it there)
            !warp_wait(&tfull_bar[buf], (n_mma / 2) & 1)) {
          fail();
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[64];
          tmem_ld_32x32b_x64(taddr0 + buf * kBN + c * 64, r);
          tmem_ld_wait_tied(*reinterpret_cast<uint32_t(*)[32]>(&r[0]));
          reg_tie32(&r[32]);
          if (c == 1 && (kSplit || kb + 1 < kb1)) {  // (the last one's place is the epilogue's)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty_bar[buf]);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float f = c == 0 || kGrad ? c0 : j / 8 < n_low ? c1 : c2;
            acc[c * 32 + j] = __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])),
                                         make_float2(f, f), acc[c * 32 + j]);
          }
        }
      }
      it += kb1 - kb0;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if constexpr (kSplit) {
        float4* srow = reinterpret_cast<float4*>(smem) + (row * kPitch + wg * kCols) / 4;
#pragma unroll
        for (int j = 0; j < kCols / 4 && row_ok; ++j)  // (rows that do not exist would meet the others' banks)
          srow[j] = make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
        continue;
      }
      // The sums go back to TMEM, where the last K block's were, and the epilogue takes them from there 16
      // columns at a time, in loops: unrolled over registers its code (16000 instructions) did not fit in the
      // instruction cache, which cost more than its arithmetic (the gradient's 24 us a tile instead of 10).
      const int m = w.row0 + row;
      const int last_buf = (n_mma - 1) & 1;
      const uint32_t tacc = taddr0 + last_buf * kBN;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(j % 2 ? acc[16 * c + j / 2].y : acc[16 * c + j / 2].x);
        tmem_st_32x32b_x32(tacc + 32 * c, r);
      }
      tmem_st_wait();
      const bool e5 = args.q_fmt == FP8GEMM_FMT_E5M2;
      if constexpr (kGrad) {
        // the thread's boxes: 4 wg .. 4 wg + 3
        const uint32_t last = it + (4 * wg + 3) / 3;
        for (uint32_t use = it + (4 * wg) / 3; use <= last && ok; ++use)
          if (!mbar_wait(&full_bar[use % kStages], (use / kStages) & 1, abort_flag, args.wait_ns)) {
            fail();
            ok = false;
          }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        auto box = [&](int b) {
          const int s = (it + b / 3) % kStages;
          return (b % 3 == 0 ? smA + s * kABytes : smB + s * kBBytes + (b % 3 - 1) * kBoxBytes) + row * 128;
        };
        const int swizzle = row & 7;
        float top_g = 0.f, top_u = 0.f;
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {  // dg to TMEM, du to the places of g and u
          uint8_t* g_row = box(4 * wg + 2 * (c / 64));
          uint8_t* u_row = box(4 * wg + 2 * (c / 64) + 1);
          uint32_t r[16];
          tmem_ld_32x32b_x16(tacc + c, r);
          tmem_ld_wait_tied16(r);
          float chunk_g = 0.f, chunk_u = 0.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint4* gp = reinterpret_cast<uint4*>(g_row + (((c % 64 / 8 + e) ^ swizzle) << 4));
            uint4* up = reinterpret_cast<uint4*>(u_row + (((c % 64 / 8 + e) ^ swizzle) << 4));
            float g[8], u[8];
            unpack8(Raw8<__nv_bfloat16>{*gp}, g);
            unpack8(Raw8<__nv_bfloat16>{*up}, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 d = swiglu_grad(__uint_as_float(r[8 * e + i]), g[i], u[i]);
              r[8 * e + i] = __float_as_uint(d.x);
              u[i] = d.y;
              chunk_g = max_nan(chunk_g, fabsf(d.x));
              chunk_u = max_nan(chunk_u, fabsf(d.y));
            }
            *gp = make_uint4(__float_as_uint(u[0]), __float_as_uint(u[1]), __float_as_uint(u[2]), __float_as_uint(u[3]));
            *up = make_uint4(__float_as_uint(u[4]), __float_as_uint(u[5]), __float_as_uint(u[6]), __float_as_uint(u[7]));
          }
          tmem_st_32x32b_x16(tacc + c, r);
          if (col + c < args.I) {
            top_g = max_nan(top_g, chunk_g);
            top_u = max_nan(top_u, chunk_u);
          }
        }
        tmem_st_wait();
        const Reciprocal sg = reciprocal(e5 ? block_scale<true>(top_g) : block_scale<false>(top_g));
        const Reciprocal su = reciprocal(e5 ? block_scale<true>(top_u) : block_scale<false>(top_u));
        const int Ip = ceil_div(args.I, kBlockK) * kBlockK;
        if (row_ok && col < args.I) {
          float* sq = args.sQ + size_t(m) * (2 * Ip / kBlockK) + col / kBlockK;
          sq[0] = sg.s;
          sq[Ip / kBlockK] = su.s;
        }
        uint8_t* q = args.Q + size_t(m) * 2 * Ip + col;
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          uint8_t* g_row = box(4 * wg + 2 * (c / 64));
          uint8_t* u_row = box(4 * wg + 2 * (c / 64) + 1);
          uint32_t r[16];
          tmem_ld_32x32b_x16(tacc + c, r);
          tmem_ld_wait_tied16(r);
          float dg[16], du[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = ((c % 64 / 8 + e) ^ swizzle) << 4;
            const float4 lo = *reinterpret_cast<const float4*>(g_row + at), hi = *reinterpret_cast<const float4*>(u_row + at);
            const float d[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dg[8 * e + i] = __uint_as_float(r[8 * e + i]);
              du[8 * e + i] = d[i];
            }
            if (args.dGU) {
              const float* v = dg + 8 * e;
              *reinterpret_cast<uint4*>(g_row + at) = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                                                                 bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
              *reinterpret_cast<uint4*>(u_row + at) = make_uint4(bf16x2_bits(d[0], d[1]), bf16x2_bits(d[2], d[3]),
                                                                 bf16x2_bits(d[4], d[5]), bf16x2_bits(d[6], d[7]));
            }
          }
          if (row_ok && col + c < args.I) {
            store_codes16(q + c, dg, sg, e5);
            store_codes16(q + Ip + c, du, su, e5);
          } else if (row_ok && col + c < Ip) {  // the rest of the last block, up to the next half
            *reinterpret_cast<uint4*>(q + c) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(q + Ip + c) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        fence_proxy_async_smem();  // before the stores and the ring's next copies
        __syncwarp();
        if (args.dGU && lane == 0) {  // the warp's 32 rows (rows and columns that do not exist are not written)
          for (int half = 0; half < 2; ++half)
            if (col + 64 * half < args.I) {
              tma_store_2d(&tmDG, box(4 * wg + 2 * half), col + 64 * half, w.row0 + (warp % 4) * 32);
              tma_store_2d(&tmDU, box(4 * wg + 2 * half + 1), col + 64 * half, w.row0 + (warp % 4) * 32);
            }
          bulk_commit_group();
          bulk_wait_group_read<0>();
        }
        if (lane == 0) mbar_arrive(gu_bar);
        it += kGuStages;
      } else {
        float top = 0.f;
#pragma unroll 2
        for (int c = 0; c < 64; c += 16) {  // h to the places of the gate values
          uint32_t g[16], u[16];
          tmem_ld_32x32b_x16(tacc + c, g);
          tmem_ld_32x32b_x16(tacc + 64 + c, u);
          tmem_ld_wait_tied16(g);
          reg_tie16(u);
          if (args.GU && row_ok && col + c < args.I) {
            __nv_bfloat16* o = args.GU + size_t(m) * 2 * args.I + col + c;
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              auto pair = [](const uint32_t* p) { return bf16x2_bits(__uint_as_float(p[0]), __uint_as_float(p[1])); };
              *reinterpret_cast<uint4*>(o + e) = make_uint4(pair(g + e), pair(g + e + 2), pair(g + e + 4), pair(g + e + 6));
              *reinterpret_cast<uint4*>(o + args.I + e) =
                  make_uint4(pair(u + e), pair(u + e + 2), pair(u + e + 4), pair(u + e + 6));
            }
          }
          __syncwarp();
          float chunk_top = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float h = swiglu(__uint_as_float(g[i]), __uint_as_float(u[i]));
            g[i] = __float_as_uint(h);
            chunk_top = max_nan(chunk_top, fabsf(h));
          }
          if (col + c < args.I) top = max_nan(top, chunk_top);
          tmem_st_32x32b_x16(tacc + c, g);
        }
        tmem_st_wait();
        // the other half of the row's block, from the thread that holds it
        float* mine = tops + (tiles & 1) * kGroups * kBlockM;
        mine[wg * kBlockM + row] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&row_bar[warp % 4]);
        ok = __all_sync(0xffffffffu, mbar_wait(&row_bar[warp % 4], tiles & 1, abort_flag, args.wait_ns));
        if (!ok) {
          fail();
          break;
        }
        top = max_nan(top, mine[(1 - wg) * kBlockM + row]);
        const Reciprocal s = reciprocal(e5 ? block_scale<true>(top) : block_scale<false>(top));
        if (row_ok && wg == 0) args.sQ[size_t(m) * ceil_div(args.I, kBlockK) + col / kBlockK] = s.s;
#pragma unroll 2
        for (int c = 0; c < 64; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tacc + c, r);
          tmem_ld_wait_tied16(r);
          float h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = __uint_as_float(r[i]);
          if (row_ok && col + c < args.I) store_codes16(args.Q + size_t(m) * args.I + col + c, h, s, e5);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[last_buf]);
    }
    if (kRingGu && lane == 0) bulk_wait_group_all();  // before this warp's shared memory can go
  } else {
    regs_decrease<kLowRegs>();  // no work: the rest of the last warpgroup
  }

  if constexpr (kSplit) {
    // every CTA of the cluster has staged its partial (or given up, and the status says so)
    __syncwarp();
    cluster_sync();
    if (warp < kPromoWarps && t_begin < total) {
      // rows of the tile shared by the cluster's CTAs, a warp for each 1x128 block; partials are
      // summed in rank order
      const GatedTile w = gated_tile<kGrad>(args, t_begin);
      const int S = args.split;
      const int r0 = part * w.rows / S, r1 = (part + 1) * w.rows / S;
      constexpr int kBlocks = kGrad ? 2 : 1;
      const float4* mine = reinterpret_cast<const float4*>(smem);
      auto sum = [&](int r, int c) {  // columns c .. c + 3 of staged row r
        const float4* p = mine + (r * kPitch + c) / 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < S; ++q) {
          const float4 x = *map_shared_rank(p, uint32_t(q));
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
        return v;
      };
      for (int i = r0 * kBlocks + warp; i < r1 * kBlocks; i += kPromoWarps) {
        const int r = i / kBlocks, blk = i % kBlocks;
        const bool e5 = args.q_fmt == FP8GEMM_FMT_E5M2;
        if constexpr (kGrad) {
          const int col = w.col0 + 128 * blk;
          if (col >= args.I) continue;
          const float4 dh = sum(r, 128 * blk + 4 * lane);
          if (e5)
            finish_dgu<true>(args, w.row0 + r, col, lane, dh);
          else
            finish_dgu<false>(args, w.row0 + r, col, lane, dh);
        } else {
          const int c = 4 * lane + 64 * (lane / 16);  // gate 0-63, up 0-63, gate 64-127, up 64-127
          const float4 g = sum(r, c), u = sum(r, c + 64);
          if (e5)
            finish_h<true>(args, w.row0 + r, w.col0, lane, g, u);
          else
            finish_h<false>(args, w.row0 + r, w.col0, lane, g, u);
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another still reads its partial
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kBN);
  }
}

// Clusters of `s` CTAs that can be resident at once (0: none).
template <bool kGrad>
int max_clusters(int dev, int s) {
  static std::atomic<int> known[64][kMaxSplit + 1] = {};  // 0 unknown, -1 none, else the count
  std::atomic<int>& k = known[dev & 63][s];
  if (k == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = s;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, gemm_gated_kernel<kGrad, true>, &cfg) != cudaSuccess) {
      cudaGetLastError();  // a refused query leaves no sticky error
      n = 0;
    }
    k = n > 0 ? n : -1;
  }
  return k > 0 ? int(k) : 0;
}

// Parts per tile when all tiles fit in one wave: as many as leave every tile's cluster resident, where that
// saves a CTA kMinSaved K blocks (half a microsecond each; the cluster's barriers and exchange cost 2 to 3 us, but its
// CTAs share the epilogue, those that are left without a K block too: 77 rows of 1040 x 400 take 9 us in 8
// parts, 12 whole; gradient of 130 rows of 400 x 272, four K blocks, 11 us in 8 parts, 14 in 4, 15 whole, 23 in 2).
constexpr int kMinSaved = 3;

template <bool kGrad>
int choose_split(const LaunchCtx& c, long long tiles, int Kb) {
  if (tiles >= c.num_sms) return 1;
  long long s = c.num_sms / tiles;
  if (s > kMaxSplit) s = kMaxSplit;
  for (; s >= 2 && Kb - ceil_div(Kb, int(s)) >= kMinSaved; --s)
    if (max_clusters<kGrad>(c.dev, int(s)) >= tiles) return int(s);
  return 1;
}

template <bool kGrad>
cudaError_t run(const LaunchCtx& c, GatedArgs a) {
  a.wait_ns = wait_limit_ns();
  CUtensorMap tmA, tmB, tmG, tmU, tmDG, tmDU;
  if (!make_tmap_u8_sw128(&tmA, a.A, uint64_t(a.M), a.K, kBlockM)) return cudaErrorInvalidValue;
  if (!make_tmap_u8_sw128(&tmB, a.B, kGrad ? uint64_t(a.I) : 2 * uint64_t(a.I), a.K, kGrad ? kBN : 64))
    return cudaErrorInvalidValue;
  memset(&tmG, 0, sizeof(tmG));
  memset(&tmU, 0, sizeof(tmU));
  memset(&tmDG, 0, sizeof(tmDG));
  memset(&tmDU, 0, sizeof(tmDU));
  if constexpr (kGrad) {  // each half on its own: what lies past it does not exist
    const uint64_t pitch = 2 * uint64_t(a.I);
    if (!make_tmap_bf16_sw128(&tmG, a.GU, a.M, a.I, pitch, kBlockM) ||
        !make_tmap_bf16_sw128(&tmU, a.GU + a.I, a.M, a.I, pitch, kBlockM))
      return cudaErrorInvalidValue;
    if (a.dGU && (!make_tmap_bf16_sw128(&tmDG, a.dGU, a.M, a.I, pitch, 32) ||
                  !make_tmap_bf16_sw128(&tmDU, a.dGU + a.I, a.M, a.I, pitch, 32)))
      return cudaErrorInvalidValue;
  }
  static SmemLimit whole, split;
  if (cudaError_t e = whole.raise(c, reinterpret_cast<const void*>(gemm_gated_kernel<kGrad, false>), kSmemBytes))
    return e;
  if (cudaError_t e = split.raise(c, reinterpret_cast<const void*>(gemm_gated_kernel<kGrad, true>), kSmemBytes))
    return e;
  const long long tiles = (long long)ceil_div(a.M, kBlockM) * ceil_div(a.I, tile_cols<kGrad>());
  if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
  a.split = choose_split<kGrad>(c, tiles, ceil_div(a.K, kBlockK));
  if (a.split == 1)
    return launch_dependent(c, gemm_gated_kernel<kGrad, false>, unsigned(tiles < c.num_sms ? tiles : c.num_sms),
                            kThreads, kSmemBytes, tmA, tmB, tmG, tmU, tmDG, tmDU, a, c.status);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(a.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_gated_kernel<kGrad, true>, tmA, tmB, tmG, tmU, tmDG, tmDU, a, c.status);
}

}  // namespace

cudaError_t launch_gemm_gated(const LaunchCtx& c, const GatedArgs& a) { return run<false>(c, a); }
cudaError_t launch_gemm_gated_backward(const LaunchCtx& c, const GatedArgs& a) { return run<true>(c, a); }

}  // namespace fp8gemm
