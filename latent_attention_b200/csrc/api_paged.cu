// Host side of the paged 8-bit latent cache: argument validation, workspace
// layout and launches of mla_paged_* and mla_decode_paged.
#include <algorithm>

#include "internal.h"
#include "paged_slices.cuh"
#include "tc.h"

namespace {

using mla::align256;
using mla::aligned16;
using mla::cuda_fail;
using mla::fail;
using mla::kMaxRequests;

// Most rows or slots of a call: row counts rounded up to whole grids stay ints.
constexpr int32_t kMaxRows = 1 << 30;

// fp32 output projection: up to this many rows a warp per output column, beyond
// the tiles of the prefill.  Whole calls of 16 heads and 2048 columns: 8 rows 20
// us for 59, 64 rows 41 for 69, 128 rows 77 for 80; of 4 heads and 256 columns: 8
// rows 14 for 25, 128 rows 19 for 31.
constexpr int kSkinnyRows = 128;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// n_blocks and block_size of a pool.
mla_status check_pool(int32_t n_blocks, int32_t block_size) {
  if (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128)
    return fail(MLA_ERR_SHAPE, "block_size=%d is not 16, 32, 64 or 128", block_size);
  if (n_blocks < 1 || (int64_t)n_blocks * block_size >= (1ll << 31))
    return fail(MLA_ERR_SHAPE, "n_blocks=%d: n_blocks x block_size must be in [1, 2^31)", n_blocks);
  return MLA_OK;
}

mla_status check_table(int32_t B, int32_t max_blocks, int32_t block_size) {
  if (B < 1 || B > kMaxRequests)
    return fail(MLA_ERR_SHAPE, "B=%d outside [1, %d]", B, kMaxRequests);
  if (max_blocks < 1 || (int64_t)max_blocks * block_size >= (1ll << 31))
    return fail(MLA_ERR_SHAPE, "max_blocks=%d: max_blocks x block_size must be in [1, 2^31)",
                max_blocks);
  return MLA_OK;
}

mla_status check_row(const mla_config& c) {
  if ((c.kv_lora_rank + c.qk_rope_head_dim) % 16)
    return fail(MLA_ERR_UNSUPPORTED,
                "paged cache rows (kv_lora_rank + qk_rope_head_dim = %d) must be a multiple of 16",
                c.kv_lora_rank + c.qk_rope_head_dim);
  return MLA_OK;
}

mla_status check_workspace(const void* ws, size_t have, size_t need) {
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(MLA_ERR_ALIGN, "workspace is not 256-byte aligned");
  if (have < need) return fail(MLA_ERR_WORKSPACE, "workspace %zu < %zu bytes", have, need);
  return MLA_OK;
}

mla::PagedPool pool_of(const mla_config& c, const void* cache, const float* scales, int n_blocks,
                       int bs) {
  mla::PagedPool p;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.scales = const_cast<float*>(scales);
  p.n_blocks = n_blocks;
  p.bs = bs;
  p.W = c.kv_lora_rank + c.qk_rope_head_dim;
  return p;
}

// Tokens per split on CUDA cores: enough splits for some sixteen blocks an SM,
// between 64 tokens (one pass of a block's threads, four a token) and 1024 (its
// partial result, r floats, stays small beside the r-byte rows that it sums).
constexpr int kSimtSplit = 1024, kSimtMinSplit = 64;
int simt_split(const mla_config& c, int64_t B, int64_t max_ctx) {
  const int64_t want = B * c.num_heads * max_ctx / (16ll * mla::device_sms());
  return (int)std::min<int64_t>(kSimtSplit, std::max<int64_t>(kSimtMinSplit, (want + 63) / 64 * 64));
}

// Partial results that the workspace holds on CUDA cores: at least B max_splits,
// and never fewer for a larger B or max_ctx (n), so that a workspace of the
// largest batch serves every smaller one.  With W = B h n / (16 SMs), B ceil(n /
// split) is at most
//   B ceil(n / 1024)                   where the split is 1024,
//   B + B n / split  otherwise, where split >= floor(W) and split >= 64, thus
//                    W / split <= 65 / 64:  B + (65 / 64) 16 SMs / h,
// and always B ceil(n / 64).
int64_t simt_parts(const mla_config& c, int64_t B, int64_t max_ctx) {
  const auto splits = [&](int64_t len) { return (max_ctx + len - 1) / len; };
  const int64_t even = B + 65ll * 16 * mla::device_sms() / (64 * c.num_heads) + 1;
  return std::max(B * splits(kSimtSplit), std::min(B * splits(kSimtMinSplit), even));
}

void paged_layout(const mla_config& c, int B, int max_blocks, int block_size,
                  mla_paged_layout* L) {
  const int64_t es = mla::elem_size(c), h = c.num_heads, r = c.kv_lora_rank;
  const int64_t w = r + c.qk_rope_head_dim;
  int64_t off = 0;
  auto take = [&](int64_t bytes) { int64_t o = off; off = align256(off + bytes); return o; };
  const int64_t max_ctx = (int64_t)max_blocks * block_size;
  L->status = take(256);
  int64_t parts;
  if (mla::tc_paged_supported(c)) {
    const mla::PagedTcPlan t = mla::tc_paged_plan(c.num_heads, mla::device_sms());
    const int64_t rows = (int64_t)B * t.groups * t.NH;
    L->split_tokens = mla::pslices::CT;
    L->max_splits = 2 * t.n_units;
    parts = L->max_splits;
    L->q_lat = -1;
    L->q8 = take(rows * 2 * w + rows * 4);     // the terms, then a factor per row
    L->plan = take(32 * (int64_t)t.n_units + ((int64_t)B + 1) * 8 + (int64_t)B * 12);
  } else {
    L->split_tokens = simt_split(c, B, max_ctx);
    L->max_splits = (int32_t)((max_ctx + L->split_tokens - 1) / L->split_tokens);
    parts = simt_parts(c, B, max_ctx);
    L->q_lat = take(B * h * w * es);
    L->q8 = L->plan = -1;
  }
  L->part_o = take(parts * h * r * 4);
  L->part_lse = take(parts * h * 4);
  L->o_lat = take(B * h * r * (mla::tc_paged_supported(c) ? 4 : es));
  // on tensor cores o is two terms for the projection behind it
  L->o = take(B * h * c.v_head_dim * es * (mla::tc_paged_supported(c) ? 2 : 1));
  L->total_bytes = off;
}

// Configuration limits of the paged decode.
mla_status check_decode(const mla_config& c, bool o_proj, int max_blocks, int block_size) {
  mla_status s = check_row(c);
  if (s != MLA_OK) return s;
  const int w = c.kv_lora_rank + c.qk_rope_head_dim;
  if (mla::tc_paged_supported(c)) {
    if (o_proj && !mla::tc_paged_oproj_supported(c))
      return fail(MLA_ERR_UNSUPPORTED, "paged decode: hidden_size=%d is not a multiple of 8",
                  c.hidden_size);
    return MLA_OK;
  }
  if (std::max(mla::paged_simt_smem(w, kSimtSplit), 4 * (c.kv_lora_rank + 256)) > mla::kMaxSmem)
    return fail(MLA_ERR_UNSUPPORTED, "paged decode: kv_lora_rank + qk_rope_head_dim = %d is too large", w);
  if ((int64_t)max_blocks * block_size > 65535ll * kSimtSplit)
    return fail(MLA_ERR_UNSUPPORTED, "paged decode: max_blocks x block_size > %lld tokens",
                65535ll * kSimtSplit);
  return MLA_OK;
}

}  // namespace

constexpr int64_t kPlanBytes = 4 * (8 + 5 * kMaxRequests);

extern "C" {

size_t mla_paged_workspace_size(int32_t n_blocks) {
  if (n_blocks < 1) return 0;
  // the status word; then the plan's prefixes or the append's bit per block
  return (size_t)align256(256 + std::max(kPlanBytes, 4 * (((int64_t)n_blocks + 31) / 32)));
}

mla_status mla_paged_plan(const int32_t* ctx_len, const int32_t* new_len, int32_t* block_table,
                          int32_t* free_ring, const int32_t* free_state, int32_t* ctx_out,
                          int32_t* free_state_out, int32_t* slot_map, int32_t* positions,
                          int32_t* cu_new, int32_t B, int32_t max_blocks, int32_t n_blocks,
                          int32_t block_size, int32_t capacity, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!ctx_len || !new_len || !block_table || !free_ring || !free_state || !ctx_out ||
      !free_state_out || !cu_new || !workspace || (capacity > 0 && !slot_map))
    return fail(MLA_ERR_NULL, "a required plan pointer is NULL");
  mla_status s = check_pool(n_blocks, block_size);
  if (s == MLA_OK) s = check_table(B, max_blocks, block_size);
  if (s != MLA_OK) return s;
  if (capacity < 0 || capacity > kMaxRows)
    return fail(MLA_ERR_SHAPE, "capacity=%d outside [0, 2^30]", capacity);
  const void* ptrs[] = {ctx_len, new_len, block_table, free_ring, free_state, ctx_out,
                        free_state_out, slot_map, positions, cu_new};
  for (const void* p : ptrs)
    if (p && !aligned4(p)) return fail(MLA_ERR_ALIGN, "pointer %p is not 4-byte aligned", p);
  s = check_workspace(workspace, workspace_bytes, 256 + kPlanBytes);
  if (s != MLA_OK) return s;
  mla::PlanArgs a{ctx_len, new_len, block_table, free_ring, free_state, ctx_out, free_state_out,
                  slot_map, positions, cu_new, B, max_blocks, n_blocks, block_size, capacity,
                  static_cast<uint32_t*>(workspace), static_cast<int32_t*>(workspace) + 64};
  const cudaError_t e = mla::launch_paged_plan(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "paged plan");
  return mla::succeed();
}

mla_status mla_paged_append(const mla_config* cfg, const void* rows, const int32_t* slot_map,
                            void* cache, float* scales, int32_t n_rows, int32_t n_blocks,
                            int32_t block_size, void* workspace, size_t workspace_bytes,
                            void* stream) {
  mla_status s = mla::check_config(cfg);
  if (s != MLA_OK) return s;
  if (!rows || !slot_map || !cache || !scales || !workspace)
    return fail(MLA_ERR_NULL, "a required append pointer is NULL");
  s = check_pool(n_blocks, block_size);
  if (s == MLA_OK) s = check_row(*cfg);
  if (s != MLA_OK) return s;
  if (n_rows < 1 || n_rows > kMaxRows)
    return fail(MLA_ERR_SHAPE, "n_rows=%d outside [1, 2^30]", n_rows);
  if (!aligned16(rows) || !aligned16(cache))
    return fail(MLA_ERR_ALIGN, "rows or cache is not 16-byte aligned");
  if (!aligned4(slot_map) || !aligned4(scales))
    return fail(MLA_ERR_ALIGN, "slot_map or scales is not 4-byte aligned");
  const size_t bits = 4 * (((size_t)n_blocks + 31) / 32);
  const size_t need = 256 + std::max<size_t>(4 * mla::kMaxStatusSlots, bits);
  s = check_workspace(workspace, workspace_bytes, need);
  if (s != MLA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  // the status word and the bit per block that claims it for one run
  if (n_rows > mla::kAppendScan) e = cudaMemsetAsync(workspace, 0, 256 + bits, st);
  if (e != cudaSuccess) return cuda_fail(e, "memset");
  uint32_t* ws = static_cast<uint32_t*>(workspace);
  e = mla::launch_paged_append(cfg->dtype, rows, slot_map, n_rows,
                               pool_of(*cfg, cache, scales, n_blocks, block_size), ws, ws + 64, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged append");
  return mla::succeed();
}

mla_status mla_paged_gather(const mla_config* cfg, const void* cache, const float* scales,
                            const int32_t* block_table, const int32_t* ctx_len, void* rows_out,
                            int32_t* cu_ctx, int32_t B, int32_t max_blocks, int32_t n_blocks,
                            int32_t block_size, int32_t capacity, void* workspace,
                            size_t workspace_bytes, void* stream) {
  mla_status s = mla::check_config(cfg);
  if (s != MLA_OK) return s;
  if (!cache || !scales || !block_table || !ctx_len || !cu_ctx || !workspace ||
      (capacity > 0 && !rows_out))
    return fail(MLA_ERR_NULL, "a required gather pointer is NULL");
  s = check_pool(n_blocks, block_size);
  if (s == MLA_OK) s = check_table(B, max_blocks, block_size);
  if (s == MLA_OK) s = check_row(*cfg);
  if (s != MLA_OK) return s;
  if (capacity < 0 || capacity > kMaxRows)
    return fail(MLA_ERR_SHAPE, "capacity=%d outside [0, 2^30]", capacity);
  if (!aligned16(cache) || !aligned16(rows_out))
    return fail(MLA_ERR_ALIGN, "cache or rows_out is not 16-byte aligned");
  if (!aligned4(scales) || !aligned4(block_table) || !aligned4(ctx_len) || !aligned4(cu_ctx))
    return fail(MLA_ERR_ALIGN, "scales, block_table, ctx_len or cu_ctx is not 4-byte aligned");
  s = check_workspace(workspace, workspace_bytes, 256 + 4 * mla::kMaxStatusSlots);
  if (s != MLA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = mla::launch_paged_gather(cfg->dtype, pool_of(*cfg, cache, scales, n_blocks, block_size),
                               block_table, ctx_len, rows_out, cu_ctx, B, max_blocks, capacity,
                               static_cast<uint32_t*>(workspace), st);
  if (e != cudaSuccess) return cuda_fail(e, "paged gather");
  return mla::succeed();
}

size_t mla_decode_paged_workspace_size(const mla_config* cfg, int32_t B, int32_t max_blocks,
                                       int32_t block_size, mla_paged_layout* layout) {
  if (mla::check_config(cfg) != MLA_OK || check_pool(1, block_size) != MLA_OK ||
      check_table(B, max_blocks, block_size) != MLA_OK ||
      check_decode(*cfg, false, max_blocks, block_size) != MLA_OK)
    return 0;
  mla_paged_layout L;
  paged_layout(*cfg, B, max_blocks, block_size, &L);
  if (layout) *layout = L;
  return (size_t)L.total_bytes;
}

mla_status mla_decode_paged(const mla_config* cfg, const void* q_nope, const void* q_pe,
                            const void* w_kv_b, const void* cache, const float* scales,
                            const int32_t* block_table, const int32_t* ctx_len, int32_t B,
                            int32_t max_blocks, int32_t n_blocks, int32_t block_size,
                            const void* w_o, void* out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  mla_status s = mla::check_config(cfg);
  if (s != MLA_OK) return s;
  const mla_config& c = *cfg;
  if (!q_nope || !q_pe || !w_kv_b || !cache || !scales || !block_table || !ctx_len || !out ||
      !workspace)
    return fail(MLA_ERR_NULL, "a required paged decode pointer is NULL");
  s = check_pool(n_blocks, block_size);
  if (s == MLA_OK) s = check_table(B, max_blocks, block_size);
  if (s == MLA_OK) s = check_decode(c, w_o != nullptr, max_blocks, block_size);
  if (s != MLA_OK) return s;
  const void* ptrs[] = {q_nope, q_pe, w_kv_b, cache, w_o, out};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return fail(MLA_ERR_ALIGN, "pointer %p is not 16-byte aligned", p);
  if (!aligned4(scales) || !aligned4(block_table) || !aligned4(ctx_len))
    return fail(MLA_ERR_ALIGN, "scales, block_table or ctx_len is not 4-byte aligned");
  mla_paged_layout L;
  paged_layout(c, B, max_blocks, block_size, &L);
  s = check_workspace(workspace, workspace_bytes, (size_t)L.total_bytes);
  if (s != MLA_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  char* ws = static_cast<char*>(workspace);
  const bool tc = mla::tc_paged_supported(c);
  cudaError_t e;
  mla::stage_event(0, st);                // the first kernel clears the status word
  mla::PagedDecodeArgs a{};
  a.q_nope = q_nope; a.q_pe = q_pe; a.w_kv_b = w_kv_b;
  a.pool = pool_of(c, cache, scales, n_blocks, block_size);
  a.table = block_table; a.ctx = ctx_len;
  a.B = B; a.max_blocks = max_blocks; a.h = c.num_heads; a.dn = c.qk_nope_head_dim;
  a.dr = c.qk_rope_head_dim; a.dv = c.v_head_dim; a.r = c.kv_lora_rank;
  a.scale = (float)mla::softmax_scale(c);
  a.split_tokens = L.split_tokens; a.max_splits = L.max_splits;
  a.q_lat = tc ? nullptr : ws + L.q_lat;
  a.part_o = (float*)(ws + L.part_o); a.part_lse = (float*)(ws + L.part_lse);
  a.o_lat = ws + L.o_lat;
  a.o = w_o ? ws + L.o : out;
  a.o_lo = w_o && tc ? ws + L.o + (int64_t)B * a.h * a.dv * 2 : nullptr;
  a.status = (uint32_t*)(ws + L.status);
  if (tc) {
    a.tc = mla::tc_paged_plan(a.h, L.max_splits / 2);
    const int64_t rows = (int64_t)B * a.tc.groups * a.tc.NH;
    a.tc.n_units = L.max_splits / 2;
    a.q8 = (uint8_t*)ws + L.q8;
    a.qf = (float*)(a.q8 + rows * 2 * (a.r + a.dr));
    a.first = (int32_t*)(ws + L.plan);
    a.pre = (int64_t*)(a.first + 8 * (int64_t)a.tc.n_units);
    a.parts = (int32_t*)(a.pre + B + 1);
    a.len = a.parts + 2 * (int64_t)B;
    e = mla::tc_paged_decode(a, st);
  } else {
    e = mla::launch_paged_decode_simt(c.dtype, a, st);
  }
  if (e != cudaSuccess) return cuda_fail(e, "paged decode");
  mla::stage_event(4, st);
  if (w_o) {
    if (tc) {
      e = mla::launch_paged_oproj(a.o, a.o_lo, w_o, out, B, a.h * a.dv, c.hidden_size, a.status, st);
    } else if (c.dtype == MLA_F32 && B <= kSkinnyRows) {
      e = mla::launch_paged_oproj_simt((const float*)a.o, (const float*)w_o, (float*)out, B,
                                       a.h * a.dv, c.hidden_size, st);
    } else {
      mla::GemmArgs go;
      go.A = a.o; go.lda = (int64_t)a.h * a.dv; go.M = B; go.K = a.h * a.dv; go.nseg = 1;
      go.Bm[0] = w_o; go.ldb[0] = (int64_t)a.h * a.dv;
      go.seg[0].out = out; go.seg[0].ldo = c.hidden_size; go.seg[0].ncols = c.hidden_size;
      e = mla::tc_gemm_supported(go, c.dtype) ? mla::tc_gemm(go, st, a.status)
                                             : mla::launch_gemm_simt(c.dtype, go, st);
    }
    if (e != cudaSuccess) return cuda_fail(e, "paged decode o_proj");
  }
  mla::stage_event(5, st);
  return mla::succeed();
}

}  // extern "C"
