// Weight-absorbed decode over the paged 8-bit latent cache on sm_100a tensor
// cores (bf16 model, latent 512 + rope 64).
//
//   P1 q_lat[b,h] = W_UK[h]^T q_nope[b,h]          batched tcgen05 GEMM
//   P2 paged_query_kernel   [q_lat | q_pe] as two e4m3 terms and a power of
//                           two per head; the chunk line of all sequences
//   P3 paged_attn_kernel    attention over the blocks (below)
//   P4 paged_combine_kernel merge of the partial results of cut sequences
//   P5 o[b,h] = W_UV[h] o_lat[b,h]                 batched tcgen05 GEMM
//
// P3.  The blocks' bytes are MMA operands as they lie in memory: no value is
// converted on the way.  What multiplies them is e4m3 too, as a sum hi + lo of
// two e4m3 terms (together 8 significant bits, bf16's precision), so a product
// takes two 8-bit MMAs, the time of one bf16 MMA, and half the bytes.
//
// Tokens are the M side, heads the N side:
//   S^T [128 tokens, 2 NH]  = C [128, 576] [Q_hi | Q_lo]^T
//   O^T [512 dims, NH]     += C^T [512, 128] P^T
// so a few heads cost no more than they should (a product with heads as M
// fills 128 rows whatever their number), C is the K-major A operand of the
// first and the MN-major A operand of the second product, and O^T of up to 64
// heads takes half of TMEM.  More than 64 heads run as equal groups, one CTA
// each, that read the same blocks at about the same time (the second reading
// comes from L2).
//
// Softmax.  A thread is a token; it holds the scores of half of the heads.
// s = raw 2^e_block f_head (log2 units); p = 2^(s - ref_head); its share of a
// row sum stays in the thread until the segment ends.  ref is the maximum of the
// segment's first chunk and moves only when a score passes it by 2^kGrow, so
// no chunk waits for O to be rescaled.  What the MMA takes is p 2^e_block
// (the bytes' own scale), which spans more than e4m3 does (a few tokens may
// hold half of the weight and thousands the rest), so every 32 tokens of a
// head carry a power of two of their own: kind::mxf8f6f4 multiplies it in
// (a ue8m0 scale per head and 32 values of K), and hi + lo keep 8 bits of
// everything within 2^-10 of the largest of the 32, nothing below 2^-18 of it.
//
// Work.  The chunks of all sequences form one line, cut into equal slices
// (paged_slices.cuh), one slice per CTA (and head group); a CTA walks its
// segments with one continuous pipeline.
//
// Warps (384 threads): 0 block lookups, L2 prefetch, TMA of the chunks (a ring
// of 128-dim boxes; one TMA load per block and box); 1 MMA issue; 2 the
// segment's query, and zeros over the rows behind a sequence's last token (a
// weight of 0 times whatever lies there could be NaN); 4-11 softmax, two
// groups of heads.  All waits are bounded; a timeout sets the status word.
#include "paged.cuh"
#include "paged_slices.cuh"
#include "sm100.cuh"
#include "tc.h"

namespace mla {
namespace {

using namespace paged;
using namespace pslices;
using namespace sm100;

constexpr int R = 512, DR = 64, W = R + DR;
constexpr int BOX = CT * 128;            // 128 tokens x 128 dims, 16 KB
constexpr int RBOX = CT * DR;            // 128 tokens x 64 rope dims, 8 KB
constexpr int NTHREADS = 384;
constexpr int PF = 3;                    // chunks looked up (and prefetched to L2) ahead
constexpr float kGrow = 24.f;

// Per head-group size NH (heads of a CTA, padded): ring depth, P buffers and
// score slots as shared memory (227 KB) and TMEM (512 columns) allow.
template <int NH>
struct Cfg {
  static constexpr int HPG = NH / 2;                       // heads per softmax group
  // both terms of P side by side (one product of N = 2 NH), or one after the
  // other (N = NH): O^T's 4 x 2 NH columns fit TMEM up to 32 heads
  static constexpr bool STK = NH <= 32;
  static constexpr int PN = STK ? 2 * NH : NH;             // columns of one O^T tile
  static constexpr int PW = STK ? 2 * NH : 64;             // bytes of a token's row of P
  static constexpr int NS = NH == 16 ? 11 : 8;             // boxes in the ring
  static constexpr int NR = NH == 64 ? 1 : 2;              // rope boxes
  static constexpr int NP = NH >= 48 ? 1 : 2;              // P buffers
  static constexpr int NSL = NH == 64 ? 1 : 2;             // score slots
  static constexpr int QBOX = 2 * NH * 128, QROPE = 2 * NH * 64, QBYTES = 4 * QBOX + QROPE;
  static constexpr int PBYTES = CT * PW * (STK ? 1 : 2);
  static constexpr int OFF_C = QBYTES;
  static constexpr int OFF_R = OFF_C + NS * BOX;
  static constexpr int OFF_P = OFF_R + NR * RBOX;
  static constexpr int OFF_SH = OFF_P + NP * PBYTES;
  static constexpr uint32_t TM_O = 0, TM_S = 4 * PN, TM_SFA = TM_S + NSL * 2 * NH,
                            TM_SFB = TM_SFA + 4;
  static constexpr int TM_COLS = TM_SFB + 4 * NP <= 256 ? 256 : 512;
};

template <int NH>
struct Shared {
  using K = Cfg<NH>;
  uint8_t sf[K::NP][512];                  // ue8m0 scales of P: head n at (n % 32) 16 + (n / 32) 4
  float hf[64], ref[64], alpha[64];        // per head: score factor, reference, O's factor
  union {
    int hmax[2][4][32];
    float lsum[2][4][32];
  };
  float scl[4][8];                         // block scales of a chunk
  uint64_t q_full, q_free, o_done, o_free, c_full[K::NS], c_empty[K::NS], r_full[K::NR],
      r_empty[K::NR], t_full[4], g_full[4], s_full[K::NSL], s_free[K::NSL], p_full[K::NP],
      pv_done[K::NP];
  uint32_t tmem_base;
  int abort_flag;
};
template <int NH>
constexpr int smem_bytes() { return Cfg<NH>::OFF_SH + (int)sizeof(Shared<NH>); }
static_assert(smem_bytes<64>() <= 227 * 1024 && smem_bytes<48>() <= 227 * 1024 &&
                  smem_bytes<32>() <= 227 * 1024 && smem_bytes<16>() <= 227 * 1024,
              "shared memory");

struct AttnParams {
  const int64_t* pre;          // [B + 1] charged chunks
  const int32_t* len;          // [B] tokens
  const int32_t* table;        // [B, max_blocks]
  const uint8_t* cache;
  const float* scales;
  const float* qf;             // [B, groups, NH]
  int B, max_blocks, n_blocks, bs, lbs;
  int h, groups, hg_heads;     // heads, head groups, heads per group
  int n_units, min_len;
  float* part_o;               // [2 n_units, h, R]
  float* part_lse;             // [2 n_units, h], log2
  __nv_bfloat16* o_lat;        // [B, h, R]
  uint32_t* status;
};

// ------------------------------------------------------------ PTX helpers
// 8-bit product, D (+)= A B^T, fp32 accumulator.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with a ue8m0 scale per row and 32 values of K of either operand.
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// 32 rows of 16 bytes into 4 TMEM columns, repeated in all four lane quarters.
__device__ __forceinline__ void tmem_cp_sf(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %1, %1, %1};" ::"r"(taddr), "r"(v)
               : "memory");
}
// Barrier `id` over `count` threads that returns the OR of their predicates.
__device__ __forceinline__ bool barrier_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
// Order of floats as order of signed integers (a positive NaN is the largest).
__device__ __forceinline__ int float_key(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_float(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
// An fp16 pair -> two e4m3 bytes, saturating.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Instruction descriptors, e4m3 operands: plain (A, B K-major), and scaled by
// ue8m0 (A, B MN-major) with the scales of K block kb in byte kb of B's column.
__host__ __device__ constexpr uint32_t idesc_f8(int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(CT >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_mxf8(int N, int kb) {
  return ((uint32_t)kb << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(CT >> 4) << 24);
}
// MN-major operand of 64- or 32-byte rows (one row per K), swizzled likewise;
// 8-row groups follow one another.
template <int ROW>
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  static_assert(ROW == 64 || ROW == 32, "row bytes");
  uint64_t d = make_desc(saddr, 16, 8 * ROW);
  d &= ~((uint64_t)7 << 61);
  return d | (uint64_t)(ROW == 64 ? 4 : 6) << 61;
}
// The scale tile: unswizzled 8-row groups of 16-byte rows.
__device__ __forceinline__ uint64_t desc_sf(uint32_t saddr) {
  uint64_t d = make_desc(saddr, 16, 128);
  return d & ~((uint64_t)7 << 61);
}
template <int ROW>
__device__ __forceinline__ uint32_t swz(uint32_t off) {
  return ROW == 64 ? off ^ (((off >> 7) & 3u) << 4) : off ^ (((off >> 7) & 1u) << 4);
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// --------------------------------------------------- P2: query and schedule
// Row (b, group, i < NH) of q8: hi at ((b G + g) 2) NH + i, lo NH rows later;
// 576 bytes each.  value = (hi + lo) 2^e with max |value| in (224, 448] 2^e.
struct QueryParams {
  const __nv_bfloat16 *q_lat, *q_pe;       // [B, h, R], [B, h, DR]
  uint8_t* q8;
  float* qf;
  const int32_t* ctx;
  int64_t* pre;
  int32_t* len;
  int B, h, groups, hg_heads, NH;
  int64_t most;                            // tokens a table holds
  float scale_log2;
  uint32_t* status;
};
constexpr int kQueryThreads = 256;

__device__ __forceinline__ void split8(const float (&v)[16], float f, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4], y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v[4 * i + k] * f;
    h[i] = to_e4m3x4(x[0], x[1], x[2], x[3]);
    from_e4m3x4(h[i], y);
    l[i] = to_e4m3x4(x[0] - y[0], x[1] - y[1], x[2] - y[2], x[3] - y[3]);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__global__ void __launch_bounds__(kQueryThreads) paged_query_kernel(QueryParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (blockIdx.x == 0) {                   // lengths and the chunk line
    __shared__ int64_t sums[kQueryThreads / 32];
    const int per = (p.B + kQueryThreads - 1) / kQueryThreads;
    const int b0 = min(t * per, p.B), b1 = min(b0 + per, p.B);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) {
      int64_t n = p.ctx[b];
      if (n < 0 || n > p.most) {
        atomicOr(p.status, kStatusBadPage);
        n = n < 0 ? 0 : p.most;
      }
      p.len[b] = (int32_t)n;
      sum += charged(n);
    }
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t at = inc - sum;
    for (int w = 0; w < warp; ++w) at += sums[w];
    for (int b = b0; b < b1; ++b) {
      at += charged(p.len[b]);
      p.pre[b + 1] = at;
    }
    if (t == 0) p.pre[0] = 0;
    return;
  }
  const int64_t row = (int64_t)(blockIdx.x - 1) * (kQueryThreads / 32) + warp;
  if (row >= (int64_t)p.B * p.groups * p.NH) return;
  const int i = (int)(row % p.NH);
  const int64_t bg = row / p.NH;
  const int g = (int)(bg % p.groups), head = g * p.hg_heads + i;
  const int64_t b = bg / p.groups;
  uint8_t* hi_row = p.q8 + (bg * 2 * p.NH + i) * W;
  uint8_t* lo_row = hi_row + (int64_t)p.NH * W;
  float v[16], r[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = 0.f;
  if (i < p.hg_heads && head < p.h) {
    load16(p.q_lat + (b * p.h + head) * R + lane * 16, v);
    const uint32_t x =
        reinterpret_cast<const uint32_t*>(p.q_pe + (b * p.h + head) * DR)[lane];
    r[0] = __uint_as_float(x << 16);
    r[1] = __uint_as_float(x & 0xffff0000u);
  }
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 18; ++k) {
    float& x = k < 16 ? v[k] : r[k - 16];
    const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
    // an infinity becomes NaN (e4m3 has none), and does not set the scale
    if (a < 0x7f800000u) amax = max(amax, a); else x = x - x;
  }
  const int e = scale_exp(__reduce_max_sync(0xffffffffu, amax));
  const float f = pow2(-e);
  uint4 hi, lo;
  split8(v, f, hi, lo);
  reinterpret_cast<uint4*>(hi_row)[lane] = hi;
  reinterpret_cast<uint4*>(lo_row)[lane] = lo;
  const uint32_t rh = to_e4m3x2(r[0] * f, r[1] * f);
  float y[4];
  from_e4m3x4(rh, y);
  reinterpret_cast<uint16_t*>(hi_row + R)[lane] = (uint16_t)rh;
  reinterpret_cast<uint16_t*>(lo_row + R)[lane] =
      (uint16_t)to_e4m3x2(r[0] * f - y[0], r[1] * f - y[1]);
  if (lane == 0) p.qf[row] = p.scale_log2 * pow2(e);
}

// ------------------------------------------------------------- P3: attention
template <int NH>
__global__ void __launch_bounds__(NTHREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmQr,
                      const __grid_constant__ CUtensorMap tmC,
                      const __grid_constant__ CUtensorMap tmCr,
                      const __grid_constant__ AttnParams p) {
  using K = Cfg<NH>;
  constexpr int HPG = K::HPG, NS = K::NS, NR = K::NR, NP = K::NP, NSL = K::NSL;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<NH>& sh = *reinterpret_cast<Shared<NH>*>(smem + K::OFF_SH);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_v = &sh.abort_flag;
  griddep_wait();
  griddep_launch_dependents();
  if (smem_u32(smem) & 1023u) {               // the swizzled tiles need it
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  const int u = blockIdx.x / p.groups, hg = blockIdx.x % p.groups;
  const Slice sl = unit_slice(p.pre, p.B, u, p.n_units, p.min_len);
  if (sl.r0 >= sl.r1) return;

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_free, 1);
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.o_free, 8);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.c_full[i], 1);
      mbar_init(&sh.c_empty[i], 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(&sh.r_full[i], 1);
      mbar_init(&sh.r_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.t_full[i], 1);
      mbar_init(&sh.g_full[i], 1);
    }
    for (int i = 0; i < NSL; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_free[i], 8);
    }
    for (int i = 0; i < NP; ++i) {
      mbar_init(&sh.p_full[i], 8);
      mbar_init(&sh.pv_done[i], 1);
    }
    sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, K::TM_COLS);
    tc_fence_before();
  }
  // scales of heads past NH are copied along with the others' and never used
  for (int i = threadIdx.x; i < NP * 512; i += NTHREADS) (&sh.sf[0][0])[i] = 127;
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sh.tmem_base;
  if (warp >= 4 && warp < 8) {                // the cache's scale is in P: A's scales are 1
    tmem_st4(tbase + ((uint32_t)((warp & 3) * 32) << 16) + K::TM_SFA, 0x7f7f7f7fu);
    tmem_wait_st();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();

  Cursor c;
  c.start(p.pre, p.B, sl, u);
  const auto advance = [&](Cursor& k) { k.next(p.pre, p.B, sl, u); };

  if (warp == 0) {
    // ---------------- lookups, L2 prefetch, the rings.  Lane i < 128 / bs has
    // the chunk's block i: its id is loaded PF + 2 chunks ahead, its scale
    // (and the block itself, into L2) PF + 1 ahead.
    if (lane == 0) {
      tma_prefetch(&tmC);
      tma_prefetch(&tmCr);
    }
    const int per_chunk = CT / p.bs;
    Cursor look = c;
    constexpr int kNone = -1;                 // no block (kNone also for ids that are refused)
    auto fetch = [&]() -> int {               // the id as the table has it; INT_MIN: no block
      int id = INT32_MIN;
      if (!look.done) {
        const int t = (look.s.c0 + look.j) * CT + lane * p.bs;
        if (lane < per_chunk && t < p.len[look.s.b]) {
          id = p.table[(int64_t)look.s.b * p.max_blocks + (t >> p.lbs)];
          if (id == INT32_MIN) id = -1;
        }
        advance(look);
      }
      return id;
    };
    auto check = [&](int id) -> int {         // a valid id, kNone without a block
      if (id == INT32_MIN) return kNone;
      if (id < 0 || id >= p.n_blocks) {
        atomicOr(p.status, kStatusBadPage);
        id = 0;
      }
      // the head groups of a unit share the prefetch
      if (lane % p.groups == hg)
        bulk_prefetch_l2(p.cache + (int64_t)id * p.bs * W, (uint32_t)(p.bs * W));
      return id;
    };
    auto scale_of = [&](int id) -> float { return id == kNone ? 1.f : p.scales[id]; };
    int ids[PF + 1], raw;
    float scs[PF + 1];
    {
      int first[PF + 2];
#pragma unroll
      for (int i = 0; i < PF + 2; ++i) first[i] = fetch();
#pragma unroll
      for (int i = 0; i < PF + 1; ++i) ids[i] = check(first[i]);
#pragma unroll
      for (int i = 0; i < PF + 1; ++i) scs[i] = scale_of(ids[i]);
      raw = first[PF + 1];
    }
    int tails = 0, g = 0, fills = 0;
    bool ok = true;
    for (; !c.done; ++g) {
      const int n = p.len[c.s.b], valid = min(CT, n - (c.s.c0 + c.j) * CT);
      const int blocks = (valid + p.bs - 1) >> p.lbs, rows = blocks << p.lbs;
      const bool tail = valid < CT;
      const int id = ids[0], y = id << p.lbs;
      // rope first: the scores start with it
      const int rs = g % NR;
      if (!warp_wait(&sh.r_empty[rs], ((g / NR) & 1) ^ 1, abort_v, p.status)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(&sh.r_full[rs], rows * DR);
      __syncwarp();
      if (lane < blocks)
        tma_load_2d(smem + K::OFF_R + rs * RBOX + (lane << p.lbs) * DR, &tmCr, R / 2, y,
                    &sh.r_full[rs]);
#pragma unroll 1
      for (int a = 0; a < 4; ++a) {
        const int f = 4 * g + a, slot = f % NS;
        if (!warp_wait(&sh.c_empty[slot], ((f / NS) & 1) ^ 1, abort_v, p.status)) { ok = false; break; }
        if (a == 0) {
          // the ring has passed chunk g - 4, whose scales lay here
          float s = scs[0];
          int e;
          if (!stored_exp(s, &e)) {
            atomicOr(p.status, kStatusBadPage);
            s = 1.f;
          }
          if (lane < 8) sh.scl[g & 3][lane] = s;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.g_full[g & 3]);
        }
        // a chunk that ends before its last row goes by way of warp 2
        uint64_t* bar = tail ? &sh.t_full[tails & 3] : &sh.c_full[slot];
        if (lane == 0) {
          if (!tail) mbar_arrive_expect_tx(bar, rows * 128);
          else if (a == 0) mbar_arrive_expect_tx(bar, 4 * rows * 128);
        }
        __syncwarp();
        if (lane < blocks)
          tma_load_2d(smem + K::OFF_C + slot * BOX + (lane << p.lbs) * 128, &tmC, 64 * a, y, bar);
        fills = f + 1;
      }
      if (!ok) break;
      if (tail) ++tails;
      advance(c);
#pragma unroll
      for (int i = 0; i < PF; ++i) {
        ids[i] = ids[i + 1];
        scs[i] = scs[i + 1];
      }
      ids[PF] = check(raw);
      scs[PF] = scale_of(ids[PF]);
      raw = fetch();
    }
    if (!ok && lane == 0) {                   // copies in flight land before the block ends
      int given_up = 0;
      for (int f = max(0, fills - NS); f < fills; ++f)
        mbar_wait(&sh.c_full[f % NS], (f / NS) & 1, &given_up, nullptr);
    }
  } else if (warp == 2) {
    // ---------------- the segment's query; zeros behind the last token
    int g0 = 0, tails = 0;
    for (; !c.done; c.next_seg(p.pre, p.B, sl, u)) {
      if (c.kk > 0 && !warp_wait(&sh.q_free, (c.kk - 1) & 1, abort_v, p.status)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.q_full, K::QBYTES);
        const int y = (c.s.b * p.groups + hg) * 2 * NH;
        tma_load_2d(smem + 4 * K::QBOX, &tmQr, R / 2, y, &sh.q_full);
        for (int a = 0; a < 4; ++a) tma_load_2d(smem + a * K::QBOX, &tmQ, 64 * a, y, &sh.q_full);
      }
      __syncwarp();
      const int valid = min(CT, p.len[c.s.b] - (c.s.c0 + c.s.nch - 1) * CT);
      g0 += c.s.nch;
      if (valid < CT) {
        if (!warp_wait(&sh.t_full[tails & 3], (tails >> 2) & 1, abort_v, p.status)) break;
        ++tails;
#pragma unroll 1
        for (int a = 0; a < 4; ++a) {
          const uint32_t box = smem_u32(smem + K::OFF_C + ((4 * (g0 - 1) + a) % NS) * BOX);
          for (int i = valid * 8 + lane; i < CT * 8; i += 32) st_shared_v4(box + i * 16, 0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0)
          for (int a = 0; a < 4; ++a) mbar_arrive(&sh.c_full[(4 * (g0 - 1) + a) % NS]);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issue: whichever of S of chunk gs (in five steps, as
    // its boxes arrive) and PV of chunk gp is ready, PV first (it frees boxes)
    if (elect_one()) {
      Cursor cs = c, cp = c;
      int gs = 0, step = 0, gp = 0;
      uint64_t t_stall = 0;
      uint32_t idle = 0;
      const uint32_t q_base = smem_u32(smem), c_base = smem_u32(smem + K::OFF_C);
      while (!cp.done) {
        bool progress = false;
        if (gp < gs && mbar_test(&sh.p_full[gp % NP], (gp / NP) & 1) &&
            (cp.j != 0 || cp.kk == 0 || mbar_test(&sh.o_free, (cp.kk - 1) & 1))) {
          tc_fence_after();
          const int pb = gp % NP;
          const uint32_t sfb = tbase + K::TM_SFB + 4 * pb;
          tmem_cp_sf(sfb, desc_sf(smem_u32(sh.sf[pb])));
          const uint64_t dp = desc_mn<K::PW>(smem_u32(smem + K::OFF_P + pb * K::PBYTES));
#pragma unroll 1
          for (int a = 0; a < 4; ++a) {
            const int slot = (4 * gp + a) % NS;
            const uint64_t dc = desc_mnmajor_sw128(c_base + slot * BOX, BOX);
#pragma unroll
            for (int term = 0; term < (K::STK ? 1 : 2); ++term)
#pragma unroll
              for (int kb = 0; kb < 4; ++kb)
                mma_mxf8(tbase + K::TM_O + a * K::PN, dc + (uint64_t)((kb * 32 * 128) >> 4),
                         dp + (uint64_t)((term * CT * 64 + kb * 32 * K::PW) >> 4),
                         idesc_mxf8(K::PN, kb), tbase + K::TM_SFA, sfb,
                         (cp.j | term | kb) != 0);
            mma_commit(&sh.c_empty[slot]);
          }
          mma_commit(&sh.pv_done[pb]);
          if (cp.j == cp.s.nch - 1) mma_commit(&sh.o_done);
          ++gp;
          advance(cp);
          progress = true;
        }
        if (!cs.done) {
          const uint32_t d = tbase + K::TM_S + (gs % NSL) * 2 * NH;
          if (step == 0) {
            if ((cs.j != 0 || mbar_test(&sh.q_full, cs.kk & 1)) &&
                (gs < NSL || mbar_test(&sh.s_free[gs % NSL], ((gs / NSL) - 1) & 1)) &&
                mbar_test(&sh.r_full[gs % NR], (gs / NR) & 1)) {
              tc_fence_after();
              const uint64_t da = desc_kmajor_sw64(smem_u32(smem + K::OFF_R + (gs % NR) * RBOX));
              const uint64_t db = desc_kmajor_sw64(q_base + 4 * K::QBOX);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                mma_f8(d, da + (uint64_t)(k * 2), db + (uint64_t)(k * 2), idesc_f8(2 * NH), k != 0);
              mma_commit(&sh.r_empty[gs % NR]);
              step = 1;
              progress = true;
            }
          } else {
            const int f = 4 * gs + step - 1, slot = f % NS;
            if (mbar_test(&sh.c_full[slot], (f / NS) & 1)) {
              tc_fence_after();
              const uint64_t da = desc_kmajor_sw128(c_base + slot * BOX);
              const uint64_t db = desc_kmajor_sw128(q_base + (step - 1) * K::QBOX);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f8(d, da + (uint64_t)(k * 2), db + (uint64_t)(k * 2), idesc_f8(2 * NH), 1);
              if (step == 4) {
                mma_commit(&sh.s_full[gs % NSL]);
                if (cs.j == cs.s.nch - 1) mma_commit(&sh.q_free);
                ++gs;
                advance(cs);
                step = 0;
              } else {
                ++step;
              }
              progress = true;
            }
          }
        }
        if (progress) {
          idle = 0;
        } else if ((++idle & 63u) == 0) {     // bounded like every other wait
          const uint64_t now = globaltimer();
          if (idle == 64) t_stall = now;
          if (*abort_v) break;
          if (now - t_stall > kWaitNs) {
            *abort_v = 1;
            atomicOr(p.status, kStatusTimeout);
            break;
          }
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------- softmax: thread = token, group = half of the heads
    const int grp = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const int h0 = grp * HPG, bar = 1 + grp;
    const int tg = (int)threadIdx.x - 128 - 128 * grp;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t p_base = smem_u32(smem + K::OFF_P);
    const int head0 = hg * p.hg_heads + h0;   // this group's first head
    const int n_heads = max(0, min(min(HPG, p.hg_heads - h0), p.h - head0));   // real ones
    bool ok = true;
    int g = 0;
    for (; !c.done; c.next_seg(p.pre, p.B, sl, u)) {
      const Seg s = c.s;
      const int n = p.len[s.b];
      if (tg < HPG) sh.hf[h0 + tg] = p.qf[((int64_t)s.b * p.groups + hg) * NH + h0 + tg];
      named_barrier_sync(bar, 128);
      float l[HPG];
#pragma unroll
      for (int i = 0; i < HPG; ++i) l[i] = 0.f;
      for (int j = 0; j < s.nch; ++j, ++g) {
        const int sls = g % NSL, pb = g % NP;
        ok = ok && warp_wait(&sh.s_full[sls], (g / NSL) & 1, abort_v, p.status) &&
             warp_wait(&sh.g_full[g & 3], (g >> 2) & 1, abort_v, p.status);
        const float sc = sh.scl[g & 3][row >> p.lbs];
        const bool live = row < n - (s.c0 + j) * CT;
        float v[HPG], us[HPG];
        {
          uint32_t a[HPG], b[HPG];
          tc_fence_after();
          const uint32_t ts = tbase + lane_off + K::TM_S + sls * 2 * NH + h0;
#pragma unroll
          for (int i = 0; i < HPG; i += 8) {
            tmem_ld8(ts + i, a + i);
            tmem_ld8(ts + NH + i, b + i);
          }
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_free[sls]);
          // raw scores of the block's values
#pragma unroll
          for (int i = 0; i < HPG; ++i)
            us[i] = (__uint_as_float(a[i]) + __uint_as_float(b[i])) * sc;
        }
        bool need = j == 0;
        if (j > 0) {
          float vm = -INFINITY;
#pragma unroll
          for (int i = 0; i < HPG; ++i) {
            v[i] = fmaf(us[i], sh.hf[h0 + i], -sh.ref[h0 + i]);
            vm = fmaxf(vm, v[i]);
          }
          need = live && vm > kGrow;
        }
        if (barrier_or(bar, 128, need || !ok)) {
          // first chunk of the segment, or a score far above its reference
          if (barrier_or(bar, 128, !ok)) { ok = false; break; }
          int mine = 0;
#pragma unroll
          for (int i = 0; i < HPG; ++i) {
            const int k = __reduce_max_sync(
                0xffffffffu, float_key(live ? us[i] * sh.hf[h0 + i] : -INFINITY));
            if (lane == i) mine = k;
          }
          if (lane < HPG) sh.hmax[grp][quad][lane] = mine;
          named_barrier_sync(bar, 128);
          if (quad == 0 && lane < HPG) {
            const float m = key_float(max(max(sh.hmax[grp][0][lane], sh.hmax[grp][1][lane]),
                                          max(sh.hmax[grp][2][lane], sh.hmax[grp][3][lane])));
            const float old = j == 0 ? m : sh.ref[h0 + lane], now = m > old ? m : old;
            sh.ref[h0 + lane] = now;
            sh.alpha[h0 + lane] = ex2(old - now);
          }
          named_barrier_sync(bar, 128);
          if (j > 0) {
            // O holds the chunks through g - 1 at the old references
            ok = warp_wait(&sh.pv_done[(g - 1) % NP], ((g - 1) / NP) & 1, abort_v, p.status);
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < HPG; ++i) l[i] *= sh.alpha[h0 + i];
#pragma unroll 1
            for (int a = 0; a < 4 * (K::STK ? 2 : 1); ++a) {
              // tile a (and its second term's columns) of this group's heads
              const uint32_t to = tbase + lane_off + K::TM_O +
                                  (K::STK ? (a >> 1) * K::PN + (a & 1) * NH : a * K::PN) + h0;
#pragma unroll
              for (int i = 0; i < HPG; i += 8) {
                uint32_t o[8];
                tmem_ld8(to + i, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  o[k] = __float_as_uint(__uint_as_float(o[k]) * sh.alpha[h0 + i + k]);
                tmem_st8(to + i, o);
              }
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int i = 0; i < HPG; ++i) v[i] = fmaf(us[i], sh.hf[h0 + i], -sh.ref[h0 + i]);
        }
        // p, its row sums, and p 2^e with a power of two per 32 tokens
        uint32_t hi[HPG / 4], lo[HPG / 4], sfb = 0;
#pragma unroll
        for (int i = 0; i < HPG; i += 4) {
          float w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float pr = live ? ex2(v[i + k]) : 0.f;
            l[i + k] += pr;
            w[k] = pr * sc;
            // the largest of the 32 (positive floats in the order of their
            // bits, NaN above all) goes to [128, 256)
            const uint32_t m = max(__reduce_max_sync(0xffffffffu, __float_as_uint(w[k])), 8u << 23);
            const uint32_t ex = m & 0x7f800000u;
            w[k] *= __uint_as_float(0x82800000u - ex);
            if (lane == i + k) sfb = (ex >> 23) - 7;
          }
          const uint32_t w01 = pack_f16(w[0], w[1]), w23 = pack_f16(w[2], w[3]);
          const uint32_t h01 = f16x2_to_e4m3x2(w01), h23 = f16x2_to_e4m3x2(w23);
          hi[i / 4] = h01 | (h23 << 16);
          lo[i / 4] = f16x2_to_e4m3x2(sub_f16x2(w01, e4m3x2_to_f16x2(h01))) |
                      (f16x2_to_e4m3x2(sub_f16x2(w23, e4m3x2_to_f16x2(h23))) << 16);
        }
        // PV of chunk g - NP has run: this buffer is free
        if (g >= NP) ok = ok && warp_wait(&sh.pv_done[pb], ((g / NP) - 1) & 1, abort_v, p.status);
        const uint32_t pt = p_base + pb * K::PBYTES;
        const uint32_t lo_at = K::STK ? NH : 0, lo_tile = K::STK ? 0 : CT * 64;
#pragma unroll
        for (int i = 0; i < HPG / 4; i += 2) {
          const uint32_t at = row * K::PW + h0 + 4 * i;
          st_shared_v2(pt + swz<K::PW>(at), hi[i], hi[i + 1]);
          st_shared_v2(pt + lo_tile + swz<K::PW>(at + lo_at), lo[i], lo[i + 1]);
        }
        if (lane < HPG) {
          const int nh = h0 + lane;
          sh.sf[pb][(nh & 31) * 16 + (nh >> 5) * 4 + quad] = (uint8_t)sfb;
          if (K::STK) sh.sf[pb][((nh + NH) & 31) * 16 + ((nh + NH) >> 5) * 4 + quad] = (uint8_t)sfb;
        }
        fence_proxy_async();
        tc_fence_before();                    // a rescaled O comes before this PV
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[pb]);
      }
      // Segment end: row sums over the 128 tokens, then the output
      if (barrier_or(bar, 128, !ok)) break;
      {
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < HPG; ++i) {
          float x = l[i];
#pragma unroll
          for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (lane == i) mine = x;
        }
        if (lane < HPG) sh.lsum[grp][quad][lane] = mine;
      }
      named_barrier_sync(bar, 128);
      ok = warp_wait(&sh.o_done, c.kk & 1, abort_v, p.status);
      tc_fence_after();
      if (ok) {
        const auto sum_of = [&](int i) {
          return (sh.lsum[grp][0][i] + sh.lsum[grp][1][i]) +
                 (sh.lsum[grp][2][i] + sh.lsum[grp][3][i]);
        };
#pragma unroll 1
        for (int i = 0; i < HPG; i += 8) {
          float inv[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) inv[k] = 1.f / sum_of(i + k);
#pragma unroll 1
          for (int a = 0; a < 4; ++a) {
            uint32_t o[8], o2[8];
            const uint32_t to = tbase + lane_off + K::TM_O + a * K::PN + h0 + i;
            tmem_ld8(to, o);
            if (K::STK) tmem_ld8(to + NH, o2);
            tmem_wait_ld();
            const int dim = a * 128 + row;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (i + k >= n_heads) continue;
              float x = __uint_as_float(o[k]);
              if (K::STK) x += __uint_as_float(o2[k]);
              x *= inv[k];
              const int head = head0 + i + k;
              if (s.whole)
                p.o_lat[((int64_t)s.b * p.h + head) * R + dim] = __float2bfloat16(x);
              else
                p.part_o[((int64_t)s.slot * p.h + head) * R + dim] = x;
            }
          }
        }
        if (!s.whole && quad == 0 && lane < n_heads)
          p.part_lse[(int64_t)s.slot * p.h + head0 + lane] =
              sh.ref[h0 + lane] + log2f(sum_of(lane));
        tc_fence_before();                    // O may be overwritten
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_free);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, K::TM_COLS);
  }
}

// P4: o_lat[b, h] of a sequence that several units hold, from their partials
// (weights 2^(lse - max)); zeros for one without tokens.  A warp per (b, h),
// 16 dims a lane.
constexpr int kCombineWarps = 4;
__global__ void __launch_bounds__(32 * kCombineWarps)
    paged_combine_kernel(const float* __restrict__ part_o, const float* __restrict__ part_lse,
                         __nv_bfloat16* __restrict__ o_lat, const int64_t* __restrict__ pre, int B,
                         int h, int n_units, int min_len) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * kCombineWarps + threadIdx.x / 32;
  if (row >= (int64_t)B * h) return;
  const int b = (int)(row / h), hh = (int)(row % h), at = (threadIdx.x % 32) * 16;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  if (pre[b + 1] != pre[b]) {
    const SeqUnits su = seq_units(pre, b, B, n_units, min_len);
    if (su.u0 == su.u1) return;            // the attention kernel wrote it
    float mx = -INFINITY;
    for (int uu = su.u0; uu <= su.u1; ++uu)
      mx = fmaxf(mx, part_lse[(int64_t)seq_slot(su, uu) * h + hh]);
    float den = 0.f;
    for (int uu = su.u0; uu <= su.u1; ++uu) {
      const int64_t part = (int64_t)seq_slot(su, uu) * h + hh;
      const float w = exp2f(part_lse[part] - mx);
      float v[16];
      load16(part_o + part * R + at, v);
      den += w;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, v[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] /= den;
  }
  store16(o_lat + row * R + at, acc);
}

template <int NH>
cudaError_t launch_attn(const AttnParams& p, const CUtensorMap& tmQ, const CUtensorMap& tmQr,
                        const CUtensorMap& tmC, const CUtensorMap& tmCr, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_attn_kernel<NH>, smem_bytes<NH>(), set);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attn_kernel<NH>, dim3(p.n_units * p.groups), dim3(NTHREADS),
                    smem_bytes<NH>(), st, tmQ, tmQr, tmC, tmCr, p);
}

}  // namespace

bool tc_paged_supported(const mla_config& c) { return tc_decode_supported(c); }

PagedTcPlan tc_paged_plan(int h, int sms) {
  PagedTcPlan t;
  t.groups = (h + 63) / 64;
  t.hg_heads = (h + t.groups - 1) / t.groups;
  t.NH = (t.hg_heads + 15) / 16 * 16;
  t.n_units = sms / t.groups > 0 ? sms / t.groups : 1;
  return t;
}

cudaError_t tc_paged_decode(const PagedDecodeArgs& a, cudaStream_t st) {
  cudaError_t e;
  const PagedTcPlan& t = a.tc;
  {
    GemmArgs g;
    g.A = a.q_nope; g.lda = (int64_t)a.h * a.dn; g.sA = a.dn; g.a_batch_inner = true;
    g.Bm[0] = a.w_kv_b; g.ldb[0] = R; g.sB = (int64_t)(a.dn + a.dv) * R; g.b_mn = true;
    g.M = a.B; g.K = a.dn; g.batch = a.h; g.nseg = 1;
    g.seg[0].out = a.q_lat; g.seg[0].ldo = (int64_t)a.h * R; g.seg[0].ncols = R;
    g.sOut = R;
    if (!tc_gemm_supported(g, MLA_BF16)) return cudaErrorNotSupported;
    e = tc_gemm(g, st, a.status);
    if (e != cudaSuccess) return e;
  }
  const int64_t rows = (int64_t)a.B * t.groups * t.NH;
  {
    QueryParams q;
    q.q_lat = (const __nv_bfloat16*)a.q_lat;
    q.q_pe = (const __nv_bfloat16*)a.q_pe;
    q.q8 = a.q8; q.qf = a.qf; q.ctx = a.ctx; q.pre = a.pre; q.len = a.len;
    q.B = a.B; q.h = a.h; q.groups = t.groups; q.hg_heads = t.hg_heads; q.NH = t.NH;
    q.most = (int64_t)a.max_blocks * a.pool.bs;
    q.scale_log2 = a.scale * 1.4426950408889634f;
    q.status = a.status;
    const int64_t per = kQueryThreads / 32;
    e = launch_pdl(paged_query_kernel, dim3((unsigned)(1 + (rows + per - 1) / per)),
                   dim3(kQueryThreads), 0, st, q);
    count_launches();
    if (e != cudaSuccess) return e;
  }
  stage_event(1, st);
  AttnParams p{};
  {
    // e4m3 tensors as pairs of bytes: 288 columns of 16 bits
    CUtensorMap tmQ, tmQr, tmC, tmCr;
    const uint64_t str[1] = {(uint64_t)W};
    const uint64_t qdims[2] = {W / 2, (uint64_t)rows * 2};
    const uint32_t qbox[2] = {64, (uint32_t)(2 * t.NH)}, qrbox[2] = {DR / 2, (uint32_t)(2 * t.NH)};
    const uint64_t cdims[2] = {W / 2, (uint64_t)a.pool.n_blocks * a.pool.bs};
    const uint32_t cbox[2] = {64, (uint32_t)a.pool.bs}, crbox[2] = {DR / 2, (uint32_t)a.pool.bs};
    if (!encode_tmap(&tmQ, a.q8, 2, qdims, str, qbox) ||
        !encode_tmap(&tmQr, a.q8, 2, qdims, str, qrbox, 64) ||
        !encode_tmap(&tmC, a.pool.cache, 2, cdims, str, cbox) ||
        !encode_tmap(&tmCr, a.pool.cache, 2, cdims, str, crbox, 64))
      return cudaErrorInvalidValue;
    p.pre = a.pre; p.len = a.len; p.table = a.table;
    p.cache = a.pool.cache; p.scales = a.pool.scales; p.qf = a.qf;
    p.B = a.B; p.max_blocks = a.max_blocks; p.n_blocks = a.pool.n_blocks; p.bs = a.pool.bs;
    p.lbs = a.pool.bs == 16 ? 4 : a.pool.bs == 32 ? 5 : a.pool.bs == 64 ? 6 : 7;
    p.h = a.h; p.groups = t.groups; p.hg_heads = t.hg_heads;
    p.n_units = t.n_units; p.min_len = 1;
    p.part_o = a.part_o; p.part_lse = a.part_lse;
    p.o_lat = (__nv_bfloat16*)a.o_lat;
    p.status = a.status;
    e = t.NH == 16   ? launch_attn<16>(p, tmQ, tmQr, tmC, tmCr, st)
        : t.NH == 32 ? launch_attn<32>(p, tmQ, tmQr, tmC, tmCr, st)
        : t.NH == 48 ? launch_attn<48>(p, tmQ, tmQr, tmC, tmCr, st)
                     : launch_attn<64>(p, tmQ, tmQr, tmC, tmCr, st);
    count_launches();
    if (e != cudaSuccess) return e;
  }
  stage_event(2, st);
  e = launch_pdl(paged_combine_kernel,
                 dim3((unsigned)(((int64_t)a.B * a.h + kCombineWarps - 1) / kCombineWarps)),
                 dim3(32 * kCombineWarps), 0, st, (const float*)a.part_o, (const float*)a.part_lse,
                 (__nv_bfloat16*)a.o_lat, (const int64_t*)a.pre, a.B, a.h, p.n_units, p.min_len);
  count_launches();
  if (e != cudaSuccess) return e;
  stage_event(3, st);
  {
    GemmArgs g;
    g.A = a.o_lat; g.lda = (int64_t)a.h * R; g.sA = R; g.a_batch_inner = true;
    g.Bm[0] = reinterpret_cast<const __nv_bfloat16*>(a.w_kv_b) + (int64_t)a.dn * R;
    g.ldb[0] = R; g.sB = (int64_t)(a.dn + a.dv) * R;
    g.M = a.B; g.K = R; g.batch = a.h; g.nseg = 1;
    g.seg[0].out = a.o; g.seg[0].ldo = (int64_t)a.h * a.dv; g.seg[0].ncols = a.dv;
    g.sOut = a.dv;
    if (!tc_gemm_supported(g, MLA_BF16)) return cudaErrorNotSupported;
    e = tc_gemm(g, st, a.status);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace mla
