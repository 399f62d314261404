// common.cuh -- definitions shared by the kernels and the host launcher.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/fp8gemm.h"

namespace fp8gemm {

constexpr int kBlockK = 128;  // K block of the scaling granularity (= 128 e4m3 bytes)
constexpr int kBlockM = 128;  // rows per tile (= TMEM lanes)
constexpr float kE4M3Max = 448.0f;

// Kernels report device-side conditions through a per-device status word
// (first error wins); the host passes its address to every launch.
__device__ __forceinline__ void raise_status(int* status, int code) {
  atomicCAS(status, 0, code);
}

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------ launch hooks
// Each kernel file exposes one host function that launches its kernels; the
// C ABI in api.cu validates arguments and then calls these.

struct LaunchCtx {
  cudaStream_t stream;
  int num_sms;
  int* status;  // device address of the status word
  int dev;      // the current device and its context's id, when the call began
  unsigned long long ctx;
};

// The quantisers; sat (device, may be null) receives the saturation count.
cudaError_t launch_quant_1x128(const LaunchCtx& c, const float* X, uint8_t* Q, float* sX,
                               int M, int K, int fmt = FP8GEMM_FMT_E4M3,
                               unsigned long long* sat = nullptr);
cudaError_t launch_quant_128x128(const LaunchCtx& c, const float* W, uint8_t* Q, float* sW,
                                 int E, int N, int K, int fmt = FP8GEMM_FMT_E4M3,
                                 unsigned long long* sat = nullptr);

// Problem description for the persistent tensor-core GEMM.
enum class GemmMode : int { kDense = 0, kContiguous = 1, kMasked = 2 };

struct GemmArgs {
  GemmMode mode;
  const uint8_t* A;
  const float* sA;
  const uint8_t* B;
  const float* sB;
  const int32_t* group_info;  // m_indices (contiguous) or masked_m (masked)
  __nv_bfloat16* D;
  int M;      // dense: M; contiguous: M_pad; masked: M_max (rows per expert)
  int N, K;
  int E;      // experts (1 for dense)
  int a_fmt = FP8GEMM_FMT_E4M3;  // operand formats (tensor-core type codes: e4m3 0, e5m2 1)
  int b_fmt = FP8GEMM_FMT_E4M3;
  // Parts per tile along K (persistent tensor-core GEMM, split instance:
  // one cluster of `split` CTAs per tile).  1: whole tiles.
  int split = 1;
  // Time limit of every pipeline wait in the kernel (the launcher fills in
  // the process-wide setting, fp8gemm_set_wait_limit_ns).
  unsigned long long wait_ns = 2000000000ull;
  // The caller's promise (FP8GEMM_FLAG_B_READ_ONLY) that no kernel still
  // running when this one starts writes B or sB: a programmatic dependent may
  // then load weights before waiting for the kernels ahead of it.
  int b_read_only = 0;
  // Persistent tensor-core GEMM: D's tensor map is valid, so whole 32-row
  // bands of a tile leave through shared memory and TMA stores.
  int d_tma = 0;
};

constexpr int kMaxSplit = 8;  // parts (cluster CTAs) per split tile, at most

// The persistent tensor-core GEMM (one launch; the count goes to *launches).
cudaError_t launch_gemm_tc(const LaunchCtx& c, const GemmArgs& a, int* launches);
// Up to FP8GEMM_MAX_DENSE_BATCH independent dense problems (host array `p`,
// validated) in one launch of the persistent tensor-core GEMM, tiles handed
// out through `counter` (two zeroed words; each launch leaves them at zero).
cudaError_t launch_gemm_tc_batch(const LaunchCtx& c, const fp8gemm_problem* p, int count,
                                 unsigned int* counter, int* launches);
// The contiguous form in expert-segment order (a one-CTA ordering kernel,
// then the persistent GEMM claiming tiles in that order): the workspace it
// needs (its counters left at zero by every launch), 0 where the form does
// not apply -- then launch_gemm_tc takes the call.
size_t contig_order_workspace_bytes(const LaunchCtx& c, const GemmArgs& a);
cudaError_t launch_gemm_tc_contiguous_ordered(const LaunchCtx& c, const GemmArgs& a, void* ws,
                                              size_t ws_bytes, int* launches);
cudaError_t launch_gemm_small_m(const LaunchCtx& c, const GemmArgs& a, void* workspace,
                                size_t workspace_bytes);
size_t small_m_workspace_bytes(int num_sms, int N);
// The dense decode path: cluster split-K where it fills the SMs (no
// workspace), stream-K through `ws` otherwise.
bool small_m_uses_workspace(const LaunchCtx& c, const GemmArgs& a);
cudaError_t launch_gemm_small_m_any(const LaunchCtx& c, const GemmArgs& a, void* ws,
                                    size_t ws_bytes);
// The dense decode path from FP32 activations X (M <= 64), quantised on load
// inside the GEMM, with Q / sA (both or neither) written too; *taken = false
// when the shape does not qualify (nothing is launched).
cudaError_t launch_gemm_small_m_quant(const LaunchCtx& c, const GemmArgs& a, const float* X,
                                      uint8_t* Q, float* sA, bool* taken);

// Many decode-sized problems from a device-resident table (gemm_table.cu),
// K split over the CTAs (stream-K) through a zeroed workspace of
// table_workspace_bytes bytes whose counters each launch leaves at zero.
size_t table_workspace_bytes(const LaunchCtx& c, int max_M);
cudaError_t launch_gemm_table(const LaunchCtx& c, const fp8gemm_problem* tab, int P, int max_M,
                              void* ws, size_t ws_bytes);

// The residual norm with FP8 output, and its gradient (norm.cu).
constexpr int kMaxNormK = 16384;

struct NormArgs {
  const void* X;
  const void* R;  // residual, or null
  const float* G;
  float eps;
  void* H;        // x + r (with R only)
  uint8_t* Q;
  float* sQ;
  float* rstd;    // or null
  int M, K;
  bool f32;       // X, R and H are FP32 rather than BF16
  int fmt;
};
cudaError_t launch_rmsnorm_quant(const LaunchCtx& c, const NormArgs& a);

struct NormGradArgs {
  const void* dY;
  const void* H;
  const float* rstd;
  const float* G;
  const void* dH;  // gradient that reaches h past the norm, or null
  void* dX;
  float* dG;
  int M, K;
  bool f32;
};
size_t rmsnorm_backward_workspace_bytes(const LaunchCtx& c);
cudaError_t launch_rmsnorm_backward(const LaunchCtx& c, const NormGradArgs& a, void* ws);

// The paged FP8 cache (kv_cache.cu, kv_attention.cu): codes
// [num_blocks, heads, block, dim], scales [num_blocks, heads].
struct KvAppendArgs {
  const __nv_bfloat16* K;  // [T, heads, dim], ld_* elements from token to token
  const __nv_bfloat16* V;
  long long ld_k, ld_v;
  uint8_t* kc;
  float* ks;
  uint8_t* vc;
  float* vs;
  const int* table;  // [B, width]
  const int* lens;   // [B]
  const int* cu;     // [B + 1], or null: T / B tokens each
  int T, B, heads, dim, block, width, num_blocks, max_new, fmt;
  int log_block;
};
cudaError_t launch_kv_append(const LaunchCtx& c, const KvAppendArgs& a);

struct KvAttentionArgs {
  const __nv_bfloat16* Q;  // [T, heads * group, dim], ld_q elements from token to token
  long long ld_q;
  const uint8_t* kc;
  const float* ks;
  const uint8_t* vc;
  const float* vs;
  const int* table;
  const int* lens;
  const int* cu;
  __nv_bfloat16* O;  // [T, heads * group, dim]
  float scale;
  int T, B, heads, group, dim, block, width, num_blocks, max_q, fmt;
  int log_block;
  unsigned long long wait_ns;  // limit of each wait for a copy
};
size_t kv_attention_workspace_bytes(const LaunchCtx& c);
cudaError_t launch_kv_attention(const LaunchCtx& c, const KvAttentionArgs& a, void* ws);

// Attention of a chunk of new tokens over the cache (kv_chunk.cu).
struct KvChunkArgs {
  const __nv_bfloat16* Q;  // [T, heads * group, dim], ld_q elements from token to token
  long long ld_q;
  const uint8_t* kc;
  const float* ks;
  const uint8_t* vc;
  const float* vs;
  const int* table;
  const int* lens;
  const int* cu;
  __nv_bfloat16* O;  // [T, heads * group, dim]
  float scale;
  int T, B, heads, group, dim, block, width, num_blocks, max_q, fmt;
  int log_block;
  bool causal;
  unsigned long long wait_ns;  // limit of each wait
  bool whole = false;          // no unit of work is split
};
size_t kv_chunk_workspace_bytes(const LaunchCtx& c);
// Whether launch_kv_attention is the kernel for a call's rows.
bool kv_chunk_few_rows(const LaunchCtx& c, const KvChunkArgs& a);
cudaError_t launch_kv_chunk(const LaunchCtx& c, const KvChunkArgs& a, void* ws, int* launches);

// The gated feed-forward products (gemm_gated.cu).
struct GatedArgs {
  const uint8_t* A;  // [M, K]: activations, or dY
  const float* sA;
  const uint8_t* B;  // W1 [2 I, K], or W2 transposed [I, K]
  const float* sB;
  uint8_t* Q;        // codes of h [M, I], or of its gradients [M, 2 Ip]
  float* sQ;
  __nv_bfloat16* GU;   // gate and up values [M, 2 I]: an output (or null), or the gradient's input
  __nv_bfloat16* dGU;  // their gradients [M, 2 I], or null
  int M, I, K, a_fmt, b_fmt, q_fmt;
  int split = 1;
  unsigned long long wait_ns = 0;
};
cudaError_t launch_gemm_gated(const LaunchCtx& c, const GatedArgs& a);
cudaError_t launch_gemm_gated_backward(const LaunchCtx& c, const GatedArgs& a);

// Rotary positions (rope.cu).
constexpr int kMaxRopeDim = 512;

struct RopeArgs {
  const void* Q;  // [T, heads_q, dim], ld_* elements from token to token
  const void* K;
  void* Qo;
  void* Ko;
  long long ld_q, ld_k, ld_qo, ld_ko;
  const float* freq;     // [rot / 2]
  const int* positions;  // [T], or null: from lens and cu
  const int* lens;       // [B]
  const int* cu;         // [B + 1], or null: T / B each
  float amplitude;
  int T, B, heads_q, heads_k, dim, rot;
  bool f32, interleaved, backward;
};
cudaError_t launch_rope(const LaunchCtx& c, const RopeArgs& a);

// The mixture-of-experts layer for a few tokens (moe_few.cu).
struct MoeArgs {
  const uint8_t* A;   // [T, H]
  const float* sA;
  const float* logits;  // [T, E]
  const uint8_t* W1;  // [E, 2 I, H]: gate rows, then up rows
  const float* s1;
  const uint8_t* W2;  // [E, H, I]
  const float* s2;
  __nv_bfloat16* D;   // [T, H]
  int* ids;           // [T, k]
  float* weights;     // [T, k]
  int T, H, I, E, k, renormalise;
  unsigned long long wait_ns;  // limit of each wait for a copy
};
size_t moe_few_workspace_bytes(const LaunchCtx& c, const MoeArgs& a);
cudaError_t launch_moe_few(const LaunchCtx& c, const MoeArgs& a, void* workspace, int* launches);

// Raises a kernel's dynamic shared memory limit, once per device and CUDA context
// (the attribute belongs to the function in one context).
struct SmemLimit {
  std::atomic<unsigned long long> set_in[64] = {};  // context id, per device
  cudaError_t raise(const LaunchCtx& c, const void* fn, size_t bytes);
};

// Launches a kernel as a programmatic dependent of the one before it on the
// stream: it may start while that one ends, and waits for it (griddepcontrol)
// before it reads or writes memory.
template <class... P, class... A>
cudaError_t launch_dependent(const LaunchCtx& c, void (*fn)(P...), dim3 grid, dim3 block,
                             size_t smem, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

// Fills `c` for the current device and `stream` (SM count, status word);
// returns an fp8gemm_status code.  Defined in api.cu.
int make_launch_ctx(cudaStream_t stream, LaunchCtx* c);
// Adds to the host-side count of kernels enqueued.  Defined in api.cu.
void count_kernel_launches(int n);
// Unique id of the calling thread's current CUDA context, 0 if none: device
// addresses cached per device are valid within one context only.  api.cu.
unsigned long long current_context_id();
// The pipeline-wait time limit kernels launched now get, in ns.  api.cu.
unsigned long long wait_limit_ns();

// Encodes a 2-D K-major uint8 tensor map with 128-byte swizzling:
// rows x cols bytes, box of box_rows x 128 bytes.  Defined in api.cu.
bool make_tmap_u8_sw128(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                        uint32_t box_rows);
// The same for rows of `cols` = 64 or 128 bytes, whole rows in a box, swizzled
// over their own length.  Defined in api.cu.
bool make_tmap_rows(CUtensorMap* map, const void* base, uint64_t rows, uint32_t cols,
                    uint32_t box_rows);
// Encodes a 2-D bf16 tensor map with 128-byte swizzling: rows x cols elements, `pitch` elements from row to
// row, box of box_rows x 64 elements (128 bytes).  False as below.  Defined in api.cu.
bool make_tmap_bf16_sw128(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t pitch,
                          uint32_t box_rows);
// Encodes a 2-D row-major bf16 tensor map with 64-byte swizzling: rows x
// cols elements, box of box_rows x 32 elements (64 bytes).  False when the
// layout cannot be described (base not 16-byte aligned, cols * 2 not a
// multiple of 16).  Defined in api.cu.
bool make_tmap_bf16_sw64(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                         uint32_t box_rows);

}  // namespace fp8gemm
