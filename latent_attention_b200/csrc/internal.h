// Internal declarations shared by the host API and the kernel launchers.
#pragma once

#include <cstdint>
#include <atomic>
#include <utility>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "mla.h"

namespace mla {

// Device status word bits (first 4 bytes of every workspace).
enum : uint32_t {
  kStatusTimeout = 1u << 0,   // a bounded wait ran out
  kStatusBadCtx = 1u << 1,    // a cu_ctx / cu_seqlens length outside its bounds
  kStatusBadPage = 1u << 2,   // paged cache: a length, block id, slot or scale out of range
  kStatusNoBlocks = 1u << 3,  // paged cache: the plan needs more blocks or slots than there are
};

// The status word stands first in a workspace.  A call that would need a launch
// of its own just to clear it leaves a word per block instead, from
// kStatusSlots (32-bit words) on, and says so in the second word: their OR is the
// status.  Every other call leaves 0 there.
constexpr uint32_t kStatusMagic = 0x5a750000u;      // | number of words
constexpr int kStatusSlots = 64, kMaxStatusSlots = 2048;

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
    return __bfloat162float(*p);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) {
    *p = __float2bfloat16_rn(v);
  }
};

// One column segment of a GEMM output and the epilogue applied to it.
// Order of operations on an fp32 accumulator value v of row m, local col n:
//   ssq_out[tile * ssq_ld + m] = sum v^2 over the tile's cols < norm_cols
//                                   (pre-gain partial, one per column tile)
//   v *= rsqrt(sum_p ssq_in[p * ssq_ld + m] * rs_inv_dim + eps)   if ssq_in
//                                   (RMS row scale; partials summed in order)
//   RoPE on cols with (n % rope_period) in [rope_start, rope_start+rope_dim)
//        position = m % T + pos_offset, pairs (i, i + rope_dim/2)  if cos
//   v *= gamma[n]                   for n < norm_cols           if gamma
//   out[m * ldo + n] = v (rounded to the element type)
struct EpiSeg {
  void* out = nullptr;
  int64_t ldo = 0;
  int ncols = 0;
  const void* gamma = nullptr;
  int norm_cols = 0;
  float* ssq_out = nullptr;
  const float* ssq_in = nullptr;
  int ssq_parts = 0;        // partial count to sum for ssq_in
  int64_t ssq_ld = 0;       // row count of the partial buffer (M)
  float rs_inv_dim = 0.f;
  float eps = 0.f;
  const float* cos = nullptr;
  const float* sin = nullptr;
  int rope_period = 0, rope_start = 0, rope_dim = 0, T = 1;
  int pos_offset = 0;       // RoPE position = (row % T) + pos_offset
  const int32_t* pos = nullptr;  // or, when set, the position of every row
  bool rope_interleave = false;  // rope columns arrive as pairs (2i, 2i+1)
};

// C = A B^T with A [M, K] (row stride lda) and the output columns split in up
// to two segments: columns of segment s come from rows of Bs [ncols_s, K].
//
// Batched products (one per attention head in decode): batch i reads
// A + i*sA, B + i*sB and writes out + i*sOut (elements).  a_batch_inner marks
// an A whose batch stride is smaller than its row stride ([rows, batch, K]
// storage).  b_mn marks a B stored [K, N] (N contiguous, row stride ldb)
// instead of nn.Linear's [N, K].
struct GemmArgs {
  const void* A = nullptr;
  int64_t lda = 0;
  const void* Bm[2] = {nullptr, nullptr};
  int64_t ldb[2] = {0, 0};
  int M = 0, K = 0;
  int nseg = 1;
  EpiSeg seg[2];
  int batch = 1;
  int64_t sA = 0, sB = 0, sOut = 0;
  bool a_batch_inner = false;
  bool b_mn = false;
};

// Causal attention of B sequences: T queries per sequence at positions
// q_off .. q_off + T - 1 against Tk keys per sequence at positions 0 .. Tk - 1
// (key j visible to query i iff j <= q_off + i).  Plain prefill: Tk = T,
// q_off = 0; prefill against a cache of T_past tokens: Tk = T_past + T,
// q_off = T_past.
struct AttnArgs {
  const void* q;        // [B*T, h, dq]
  const void* kv;       // [B*Tk, h, dn+dv]
  const void* ckv;      // [B*Tk, r_kv+dr]  (k_pe at column r_kv)
  void* o;              // [B*T, h, dv]
  int B, T, h, dn, dr, dv, r_kv;
  float scale;
  uint32_t* status;
  int Tk = 0, q_off = 0;
  // Packed (THD) prefill: sequence b owns rows cu_seqlens[b] .. cu_seqlens[b+1]-1
  // of `total` rows; B is the sequence count and T the longest sequence.
  const int32_t* cu_seqlens = nullptr;
  int total = 0;
};

struct DecodeArgs {
  const void* q_nope;   // [B, h, dn]
  const void* q_pe;     // [B, h, dr]
  const void* w_kv_b;   // [h*(dn+dv), r]
  const void* cache;    // [sum ctx, r + dr]
  const int32_t* cu_ctx;
  int B, max_ctx, h, dn, dr, dv, r;
  float scale;
  int split_tokens, max_splits;   // SIMT path: tokens per split, splits per sequence
  int n_units, min_len;           // tensor-core path: CTA pairs, shortest slice
  void* q_lat;          // [B, h, r + dr]
  float* part_o;        // SIMT [B, max_splits, h, r]; tensor cores [2 n_units, h, r]
  float* part_lse;      // SIMT [B, max_splits, h];    tensor cores [2 n_units, h]
  void* o_lat;          // [B, h, r]
  void* o;              // [B, h, dv]
  uint32_t* status;
};

// The paged 8-bit latent cache (mla_paged_*): a pool of n_blocks blocks of bs
// rows of W = r + dr e4m3 values, one power-of-two scale per block.
struct PagedPool {
  uint8_t* cache;       // [n_blocks, bs, W]
  float* scales;        // [n_blocks]
  int n_blocks, bs, W;
};

struct PlanArgs {
  const int32_t *ctx, *fresh;      // [B] cached tokens; new tokens or -1
  int32_t *table, *ring;           // [B, max_blocks], [n_blocks]
  const int32_t* state;            // {head, count} of the ring
  int32_t *ctx_out, *state_out, *slots, *pos, *cu;
  int B, max_blocks, n_blocks, bs, capacity;
  uint32_t* status;
  int32_t* sums;                   // [8 + 5 B]: the prefixes, where a second grid needs them
};

// SMs of a B200: what the paged launch rules count with (and were measured on).
constexpr int kSMs = 148;

// Requests a paged call takes at most: every scan over them fits the shared
// memory of one block.
constexpr int kMaxRequests = 8192;

// Tensor-core paged decode: the heads in `groups` equal groups of hg_heads
// (padded to NH), n_units slices of the tokens per group.
struct PagedTcPlan {
  int groups, hg_heads, NH, n_units;
};

// Weight-absorbed decode over the pool's blocks.
struct PagedDecodeArgs {
  const void *q_nope, *q_pe, *w_kv_b;
  PagedPool pool;
  const int32_t *table, *ctx;      // [B, max_blocks], [B]
  int B, max_blocks, h, dn, dr, dv, r;
  float scale;
  int split_tokens, max_splits;    // CUDA cores: tokens per split, splits per sequence
  void* q_lat;                     // [B, h, r + dr]
  float *part_o, *part_lse;        // [B, max_splits, h, r], [B, max_splits, h]
  void* o_lat;                     // [B, h, r]
  void* o;                         // [B, h, dv]
  void* o_lo;                      // tensor cores: its second term, or null
  uint32_t* status;
  // tensor cores: no q_lat, o_lat in fp32, the partials [2 n_units, h, ...]
  PagedTcPlan tc;
  uint8_t* q8;                     // [B, groups, 2, NH, r + dr] e4m3 terms
  float* qf;                       // [B, groups, NH]
  int64_t* pre;                    // [B + 1]
  int32_t *len, *first, *parts;    // [B]; [n_units][8] a unit's first segment; [B][2] partials
};

// cudaFuncSetAttribute applies to the current device only: set a kernel's
// dynamic shared-memory limit once per device (devices 0..63).
inline cudaError_t set_dynamic_smem(const void* kernel, int bytes,
                                    std::atomic<uint64_t>& done_devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit && (done_devices.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done_devices.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches a kernel with programmatic stream serialization: it may start
// (prologue: barriers, TMEM, descriptor prefetch) while the previous kernel
// of the stream finishes.  Only for kernels that call griddep_wait() first
// (see sm100.cuh).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Launch accounting and stage events (defined in api.cu).
void count_launches(int n = 1);
// Sets the text mla_last_error_detail() returns on this host thread.
void set_error_detail(const char* msg);
// Records registered stage event i (if any) on stream st.
void stage_event(int i, cudaStream_t st);
// Host checks and sizes shared by the entry points (defined in api.cu): an
// error status with its detail text, the configuration's self-checks, the
// softmax scale, the SM count of the current device.
mla_status fail(mla_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mla_status cuda_fail(cudaError_t e, const char* what);
mla_status succeed();
mla_status check_config(const mla_config* c);
double softmax_scale(const mla_config& c);
int device_sms();
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }
inline int elem_size(const mla_config& c) { return c.dtype == MLA_F32 ? 4 : 2; }

// Launchers (return the launch error).
cudaError_t launch_rope_tables(const mla_config& cfg, int max_pos, float* cos,
                               float* sin, cudaStream_t st);
cudaError_t launch_gemm_simt(int dtype, const GemmArgs& a, cudaStream_t st);
// Column tile width of the CUDA-core GEMM (RMS partial count = ceil(cols/64)).
constexpr int kSimtTileN = 64;
cudaError_t launch_attn_simt(int dtype, const AttnArgs& a, cudaStream_t st);
// Normalised latent rows [RMSNorm(c) | k_pe] from the gain-scaled latent
// buffer: source row m (of N = B*T) goes to destination row
// (m / T) * dst_T + dst_off + (m % T).
// Packed prefill: pos[m] = m - cu_seqlens[b(m)] for the `total` packed rows;
// malformed cu_seqlens raise kStatusBadCtx (positions stay in [0, max_len)).
cudaError_t launch_packed_positions(const int32_t* cu_seqlens, int n_seq, int total, int max_len,
                                    int32_t* pos, uint32_t* status, cudaStream_t st);

cudaError_t launch_latent_finalize(int dtype, const void* ckv,
                                   const float* ssq_kv, int ssq_parts, int N, int r_kv,
                                   int dr, float eps, void* cache,
                                   cudaStream_t st, int T = 1, int dst_T = 1, int dst_off = 0);
cudaError_t launch_decode_simt(int dtype, const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st);
// Rows up to which an append finds a block's second run by looking through the
// slots before it; beyond, a bit per block (claims, zeroed with the status by a
// memset of its own) tells.  Around 4000 rows in runs of 64 the look takes 5.5 us
// for 8.3 with the bits, in runs of one 12.4 for 10.9; around 8000, 8.2 for 10.4
// and (6000) 21.4 for 16.4.
constexpr int kAppendScan = 4096;
cudaError_t launch_paged_append(int dtype, const void* rows, const int32_t* slots, int n_rows,
                                const PagedPool& pool, uint32_t* status, uint32_t* claims,
                                cudaStream_t st);
cudaError_t launch_paged_gather(int dtype, const PagedPool& pool, const int32_t* table,
                                const int32_t* ctx, void* rows, int32_t* cu, int B,
                                int max_blocks, int capacity, uint32_t* status, cudaStream_t st);
// Shared memory of the CUDA-core paged decode: the query, 1024 partial sums,
// the split's scores and, per 16 tokens, a scale and a block id.
constexpr int kMaxSmem = 227 * 1024 - 1024;
inline int paged_simt_smem(int w, int split_tokens) {
  return 4 * (w + 1024 + split_tokens + 2 * (split_tokens / 16));
}
cudaError_t launch_paged_oproj_simt(const float* o, const float* w_o, float* out, int B, int K,
                                    int hidden, cudaStream_t st);
cudaError_t launch_paged_decode_simt(int dtype, const PagedDecodeArgs& a, cudaStream_t st);
// Smallest workspace mla_decode_absorbed runs with (one SM pair on tensor cores).
size_t decode_min_workspace(const mla_config& c, int B, int max_ctx);

}  // namespace mla
