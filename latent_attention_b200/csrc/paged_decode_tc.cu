// Weight-absorbed decode over the paged 8-bit latent cache on sm_100a tensor
// cores (bf16 model, latent 512 + rope 64).
//
//   P1 paged_query_kernel   q_lat = W_UK^T q_nope; [q_lat | q_pe] as two e4m3
//                           terms and a power of two per head (paged_proj.cu)
//   P2 paged_attn_kernel    attention over the blocks (below)
//   P3 paged_output_kernel  merge of the partial results of cut sequences,
//                           o = W_UV o_lat (paged_proj.cu)
//
// P2.  The blocks' bytes are MMA operands as they lie in memory: no value is
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
// Softmax.  A thread is a token; it holds the scores of 16 heads.
// s = raw 2^e_block f_head (log2 units); p = 2^(s - ref_head); its share of a
// row sum stays in the thread until the segment ends.  ref is the score of
// the segment's first token and moves only when a score passes it by kGrow
// (to the chunk's maximum), so hardly a chunk waits for O to be rescaled.  What
// the MMA takes is p 2^e_block (the bytes' own scale), which spans more than
// e4m3 does (a few tokens may hold half of the weight and thousands the rest),
// so every 32 tokens of a head carry a power of two of their own:
// kind::mxf8f6f4 multiplies it in (a ue8m0 scale per head and 32 values of K),
// and hi + lo keep 8 bits of everything within 2^-10 of the largest of the 32,
// nothing below 2^-18 of it.
//
// Work.  The chunks of all sequences form one line, cut into equal slices
// (paged_slices.cuh), one slice per CTA (and head group); a CTA walks its
// segments with one continuous pipeline.
//
// Warps: 0 and 2 TMA of the chunks (a ring of 128-dim boxes; one load per block
// and box), 2 also the block lookups; 1 the segments' queries and the MMAs of S;
// 3 the MMAs of PV; from 4 on softmax, groups of 16 (8) heads.  S and PV have a
// thread each so that neither waits for the other's inputs: PV of a chunk frees
// the boxes of the next but one.  All waits are bounded; a timeout sets the
// status word.
//
// Measured (whole calls of 64 sequences of 16384 tokens in blocks of 64, at an SM
// clock of 1965 MHz): 128 heads 334 us, 1.7 PFLOP/s executed in 8 bits; 64 heads
// 186 us; 16 heads 132 us, 4.6 TB/s.  Kept up for a second, the power cap takes the
// clock to 1.66 GHz: 380, 205 and 132 us.  What bounds it: shared memory holds two
// chunks at 64 heads (2.75 at 16), and a chunk stays from its load's issue until
// PV frees it, some 3000 cycles of load, 2000-3000 of S, 2000 of softmax and
// 1500-2500 of PV.  The MMAs of 64 heads take 2280 cycles a chunk of the 4200
// (their A operand comes from shared memory at 128 bytes a cycle, which the
// collector halves for PV's second term); at 16 heads loads alone, without MMAs
// or softmax, take 121 us of 131 between events.  Leaving out PV, S, loads or
// exponentials alone gave 268, 274, 295 and 285 us of 295 at 128 heads.
// Measured and not kept: two sets of softmax warps on alternate chunks (377 us
// for 291), four loading warps (16 heads 2 % faster, 48 heads 9 % slower for
// want of registers), waits by one lane or without a pause between tries (5-10 %
// slower), blocks' lines asked for ahead in L2 (the same).
#include "paged.cuh"
#include "paged_slices.cuh"
#include "ring_drain.cuh"
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
constexpr int GR = 6;                    // lookup ring, chunks
constexpr int AHEAD = 3;                 // chunks looked up ahead of loads
constexpr float kGrow = 24.f;

// Per head-group size NH (heads of a CTA, padded): ring depth, P buffers and
// score slots as shared memory (227 KB) and TMEM (512 columns) allow.
template <int NH>
struct Cfg {
  static constexpr int HPG = NH == 16 ? 8 : 16;            // heads per softmax group
  static constexpr int NG = NH / HPG, NTHREADS = 128 + 128 * NG;
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
  float hf[64], nref[64], alpha[64];       // per head: score factor, -reference, factor of O
  union {                                  // per warp and head; barriers part the uses
    float inv[K::NG][4][K::HPG];           // 2^-k of its P
    int hmax[K::NG][4][K::HPG];
    float lsum[K::NG][4][K::HPG];
  };
  float scl[GR][8];                        // scales and ids of a chunk's blocks
  int ids[GR][8];
  uint64_t q_full, q_free, o_done, o_free, c_full[K::NS], c_empty[K::NS], r_full[K::NR],
      r_empty[K::NR], g_full[GR], e_full[GR], s_full[K::NSL], s_free[K::NSL],
      p_full[K::NP], pv_done[K::NP];
  uint32_t tmem_base;
  int abort_flag;
  int issued[4];                           // ring positions filled: boxes (warp 0, warp 2), rope, queries
};
template <int NH>
constexpr int smem_bytes() { return Cfg<NH>::OFF_SH + (int)sizeof(Shared<NH>); }
static_assert(smem_bytes<64>() <= 227 * 1024 && smem_bytes<48>() <= 227 * 1024 &&
                  smem_bytes<32>() <= 227 * 1024 && smem_bytes<16>() <= 227 * 1024,
              "shared memory");

struct AttnParams {
  const int64_t* pre;          // [B + 1] charged chunks
  const int32_t* len;          // [B] tokens
  const int4* first;           // [n_units][2] a unit's first segment: b, c0, nch, slot; whole, tokens
  const int32_t* table;        // [B, max_blocks]
  const float* scales;
  const float* qf;             // [B, groups, NH]
  int B, max_blocks, n_blocks, bs, lbs;
  int h, groups, hg_heads;     // heads, head groups, heads per group
  int n_units, min_len;
  float* part_o;               // [2 n_units, h, R]
  float* part_lse;             // [2 n_units, h], log2
  float* o_lat;                // [B, h, R], sequences in one segment
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
// A may stay in the tensor core's collector for the next product with it
// (KEEP: fill) or come from there (USE: last use), which saves reading it.
enum Collector { NONE, KEEP, USE };
template <Collector C>
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t acc) {
  if (C == KEEP)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X.collector::a::fill "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else if (C == USE)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X.collector::a::lastuse "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
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
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t* r) {
  static_assert(N == 8 || N == 16, "columns");
  if (N == 8) tmem_ld8(taddr, r); else tmem_ld16(taddr, r);
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

// After an abort: the copies still in flight (boxes by warps 0 and 2, rope,
// queries) land before the block leaves its shared memory.  (Out of line: inlined
// it moved other code, and 64 heads took 335 us for 325.)
template <int NH>
__device__ __noinline__ void drain(Shared<NH>& sh) {
  using K = Cfg<NH>;
  int given_up = 0;
  const auto wait = [&](uint64_t* full) {
    return [=, &given_up](int slot, uint32_t parity) {
      mbar_wait(&full[slot], parity, &given_up, nullptr);
    };
  };
  const int i0 = sh.issued[0], i2 = sh.issued[1];
  drain_ring(max(i0, i2), K::NS, [=](int f) { return f < ((f & 3) < 2 ? i0 : i2); },
             wait(sh.c_full));
  drain_ring(sh.issued[2], K::NR, [](int) { return true; }, wait(sh.r_full));
  drain_ring(sh.issued[3], 1, [](int) { return true; }, wait(&sh.q_full));
}

// ------------------------------------------------------------- P2: attention
template <int NH>
__global__ void __launch_bounds__(Cfg<NH>::NTHREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmQr,
                      const __grid_constant__ CUtensorMap tmC,
                      const __grid_constant__ CUtensorMap tmCr,
                      const __grid_constant__ AttnParams p) {
  using K = Cfg<NH>;
  constexpr int HPG = K::HPG, NS = K::NS, NR = K::NR, NP = K::NP, NSL = K::NSL, NG = K::NG;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<NH>& sh = *reinterpret_cast<Shared<NH>*>(smem + K::OFF_SH);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_v = &sh.abort_flag;
  if (smem_u32(smem) & 1023u) {               // the swizzled tiles need it
    griddep_wait();
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  const int u = blockIdx.x / p.groups, hg = blockIdx.x % p.groups;

  // what needs nothing of the kernel before this one
  if (warp == 0) {
    if (lane == 0) {
      mbar_init(&sh.q_full, 1);
      mbar_init(&sh.q_free, 1);
      mbar_init(&sh.o_done, 1);
      mbar_init(&sh.o_free, 4 * NG);
      for (int i = 0; i < NS; ++i) {
        mbar_init(&sh.c_full[i], 1);
        mbar_init(&sh.c_empty[i], 1);
      }
      for (int i = 0; i < NR; ++i) {
        mbar_init(&sh.r_full[i], 1);
        mbar_init(&sh.r_empty[i], 1);
      }
      for (int i = 0; i < GR; ++i) {
        mbar_init(&sh.g_full[i], 1);
        mbar_init(&sh.e_full[i], 1);
      }
      for (int i = 0; i < NSL; ++i) {
        mbar_init(&sh.s_full[i], 1);
        mbar_init(&sh.s_free[i], 4 * NG);
      }
      for (int i = 0; i < NP; ++i) {
        mbar_init(&sh.p_full[i], 4 * NG);
        mbar_init(&sh.pv_done[i], 1);
      }
      sh.abort_flag = 0;
      fence_barrier_init();
    }
  } else if (warp == 1) {
    tmem_alloc(&sh.tmem_base, K::TM_COLS);
    tc_fence_before();
  } else if (warp == 3 && lane == 0) {
    tma_prefetch(&tmC);
    tma_prefetch(&tmCr);
    tma_prefetch(&tmQ);
    tma_prefetch(&tmQr);
  }
  // scales of heads past NH are copied along with the others' and never used
  for (int i = threadIdx.x; i < NP * 512; i += K::NTHREADS) (&sh.sf[0][0])[i] = 127;
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
  griddep_wait();
  griddep_launch_dependents();
  Cursor c;                                   // (done at once where the slice is empty)
  const int4 f0 = p.first[2 * u], f1 = p.first[2 * u + 1];
  const int64_t total = p.pre[p.B];           // (the slice itself matters from the second segment on)
  {
    Seg s;
    s.b = f0.x; s.c0 = f0.y; s.nch = f0.z; s.slot = f0.w;
    s.whole = f1.x != 0;
    c.resume(s);
  }
  const int n_first = f1.y;                   // tokens of its sequence
  Slice sl;
  sl.r0 = imin(u * slice_len(total, p.n_units, p.min_len), total);
  sl.r1 = imin(sl.r0 + slice_len(total, p.n_units, p.min_len), total);
  const auto tokens = [&](const Cursor& k) { return k.kk == 0 ? n_first : p.len[k.s.b]; };
  const auto advance = [&](Cursor& k) { k.next(p.pre, p.B, sl, u); };

  // TMA loads of box a of a chunk's `blocks` blocks (ids in shared memory); a
  // thread issues one in some 90 cycles, so two warps share them
  const auto load_box = [&](int a, int slot, int blocks, const int* ids) {
    mbar_arrive_expect_tx(&sh.c_full[slot], (blocks << p.lbs) * 128);
    for (int i = 0; i < blocks; ++i)
      tma_load_2d(smem + K::OFF_C + slot * BOX + (i << p.lbs) * 128, &tmC, 64 * a, ids[i] << p.lbs,
                  &sh.c_full[slot]);
  };
  if (warp == 0) {
    // ---------------- TMA of the rope boxes and of the first two boxes
    if (elect_one()) {
      int slot = 0, rs = 0, g = 0, n = 0;
      int issued = 0, ropes = 0;              // ring positions behind this warp's last loads
      uint32_t ph = 1, rph = 1;               // parities of the empty barriers
      for (; !c.done; ++g) {
        if (c.j == 0) n = tokens(c);
        const int valid = min(CT, n - (c.s.c0 + c.j) * CT);
        const int blocks = (valid + p.bs - 1) >> p.lbs;
        if (!mbar_wait(&sh.g_full[g % GR], (g / GR) & 1, abort_v, p.status)) break;
        const int* ids = sh.ids[g % GR];
        // rope first: the scores start with it
        if (!mbar_wait(&sh.r_empty[rs], rph, abort_v, p.status)) break;
        mbar_arrive_expect_tx(&sh.r_full[rs], (blocks << p.lbs) * DR);
        for (int i = 0; i < blocks; ++i)
          tma_load_2d(smem + K::OFF_R + rs * RBOX + (i << p.lbs) * DR, &tmCr, R / 2,
                      ids[i] << p.lbs, &sh.r_full[rs]);
        ++ropes;
        if (++rs == NR) { rs = 0; rph ^= 1; }
        if (!mbar_wait(&sh.c_empty[slot], ph, abort_v, p.status)) break;
        load_box(0, slot, blocks, ids);
        issued = 4 * g + 1;
        if (++slot == NS) { slot = 0; ph ^= 1; }
        if (!mbar_wait(&sh.c_empty[slot], ph, abort_v, p.status)) break;
        load_box(1, slot, blocks, ids);
        issued = 4 * g + 2;
        slot += 3;
        if (slot >= NS) { slot -= NS; ph ^= 1; }
        advance(c);
      }
      sh.issued[0] = issued;
      sh.issued[2] = ropes;
    }
  } else if (warp == 1) {
    // ---------------- the segments' queries, S of every chunk
    if (elect_one()) {
      int slot = 0, rs = 0, g = 0, queries = 0;
      uint32_t ph = 0, rph = 0;
      const uint32_t qb = smem_u32(smem);
      const uint64_t dq = desc_kmajor_sw128(qb), dqr = desc_kmajor_sw64(qb + 4 * K::QBOX);
      const uint64_t dc0 = desc_kmajor_sw128(smem_u32(smem + K::OFF_C));
      const uint64_t dr0 = desc_kmajor_sw64(smem_u32(smem + K::OFF_R));
      for (bool ok = true; ok && !c.done; ++g) {
        if (c.j == 0) {
          if (c.kk > 0 && !mbar_wait(&sh.q_free, (c.kk - 1) & 1, abort_v, p.status)) break;
          mbar_arrive_expect_tx(&sh.q_full, K::QBYTES);
          const int y = (c.s.b * p.groups + hg) * 2 * NH;
          tma_load_2d(smem + 4 * K::QBOX, &tmQr, R / 2, y, &sh.q_full);
          for (int a = 0; a < 4; ++a) tma_load_2d(smem + a * K::QBOX, &tmQ, 64 * a, y, &sh.q_full);
          ++queries;
          if (!mbar_wait(&sh.q_full, c.kk & 1, abort_v, p.status)) break;
        }
        const int sls = g % NSL;
        const uint32_t d = tbase + K::TM_S + sls * 2 * NH;
        if (g >= NSL && !mbar_wait(&sh.s_free[sls], ((g / NSL) - 1) & 1, abort_v, p.status)) break;
        if (!mbar_wait(&sh.r_full[rs], rph, abort_v, p.status)) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 2; ++k)
          mma_f8(d, dr0 + (uint64_t)((rs * RBOX + k * 32) >> 4), dqr + (uint64_t)(k * 2),
                 idesc_f8(2 * NH), k != 0);
        mma_commit(&sh.r_empty[rs]);
        if (++rs == NR) { rs = 0; rph ^= 1; }
#pragma unroll 1
        for (int a = 0; a < 4; ++a) {
          if (!mbar_wait(&sh.c_full[slot], ph, abort_v, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint64_t da = dc0 + (uint64_t)((slot * BOX) >> 4);
          const uint64_t db = dq + (uint64_t)((a * K::QBOX) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f8(d, da + (uint64_t)(k * 2), db + (uint64_t)(k * 2), idesc_f8(2 * NH), 1);
          if (++slot == NS) { slot = 0; ph ^= 1; }
        }
        if (!ok) break;
        mma_commit(&sh.s_full[sls]);
        if (c.j == c.s.nch - 1) mma_commit(&sh.q_free);
        advance(c);
      }
      sh.issued[3] = queries;
    }
  } else if (warp == 3) {
    // ---------------- PV of every chunk
    if (elect_one()) {
      int slot = 0, g = 0;
      const uint64_t dc0 = desc_mnmajor_sw128(smem_u32(smem + K::OFF_C), BOX);
      const uint64_t dp0 = desc_mn<K::PW>(smem_u32(smem + K::OFF_P));
      const uint64_t dsf = desc_sf(smem_u32(sh.sf[0]));
      for (; !c.done; ++g) {
        const int pb = g % NP;
        if (c.j == 0 && c.kk > 0 && !mbar_wait(&sh.o_free, (c.kk - 1) & 1, abort_v, p.status))
          break;
        if (!mbar_wait(&sh.p_full[pb], (g / NP) & 1, abort_v, p.status)) break;
        tc_fence_after();
        const uint32_t sfb = tbase + K::TM_SFB + 4 * pb;
        tmem_cp_sf(sfb, dsf + (uint64_t)((pb * 512) >> 4));
        const uint64_t dp = dp0 + (uint64_t)((pb * K::PBYTES) >> 4);
        const uint32_t keep = c.j != 0;
#pragma unroll 1
        for (int a = 0; a < 4; ++a) {
          const uint64_t dc = dc0 + (uint64_t)((slot * BOX) >> 4);
#pragma unroll
          for (int kb = 0; kb < 4; ++kb) {
            const uint32_t to = tbase + K::TM_O + a * K::PN, sfa = tbase + K::TM_SFA;
            const uint64_t da = dc + (uint64_t)((kb * 32 * 128) >> 4);
            const uint64_t db = dp + (uint64_t)((kb * 32 * K::PW) >> 4);
            const uint32_t id = idesc_mxf8(K::PN, kb), acc = kb ? 1u : keep;
            if (K::STK) {
              mma_mxf8<NONE>(to, da, db, id, sfa, sfb, acc);
            } else {
              mma_mxf8<KEEP>(to, da, db, id, sfa, sfb, acc);
              mma_mxf8<USE>(to, da, db + (uint64_t)((CT * 64) >> 4), id, sfa, sfb, 1);
            }
          }
          mma_commit(&sh.c_empty[slot]);
          if (++slot == NS) slot = 0;
        }
        mma_commit(&sh.pv_done[pb]);
        if (c.j == c.s.nch - 1) mma_commit(&sh.o_done);
        advance(c);
      }
    }
  } else if (warp == 2) {
    // ---------------- lookups, and TMA of the last two boxes.  Lane i <
    // 128 / bs looks up block i of a chunk, AHEAD chunks before its loads; the
    // id of one chunk is loaded while the scale of the one before is.
    const int per_chunk = CT / p.bs;
    Cursor look = c;
    int ln = 0, n = 0, lg = 0;
    auto fetch = [&]() -> int {               // the id as the table has it; INT_MIN: no block
      int id = INT32_MIN;
      if (!look.done) {
        if (look.j == 0) ln = tokens(look);
        const int t = (look.s.c0 + look.j) * CT + lane * p.bs;
        if (lane < per_chunk && t < ln) {
          id = p.table[(int64_t)look.s.b * p.max_blocks + (t >> p.lbs)];
          if (id == INT32_MIN) id = -1;
        }
      }
      return id;
    };
    int id = fetch();
    // Entry lg % GR was chunk lg - GR's = g - 3 of the chunk g just loaded,
    // whose last box has waited for a box of chunk g - 2 (the ring holds less
    // than three chunks): every softmax warp is past g - 3.
    // Every load is used one call later, so that no call waits for one.
    float sc = 1.f;                           // the scale of entry lg - 1
    bool pending = false;
    auto look_up = [&]() {
      if (pending) {
        const int at = (lg - 1) % GR;
        sc = read_scale(sc, p.status);
        if (lane < 8) sh.scl[at][lane] = sc;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.e_full[at]);
      }
      pending = !look.done;
      if (!pending) return;
      const int at = lg % GR;
      const bool has = id != INT32_MIN;
      if (has && (id < 0 || id >= p.n_blocks)) {
        atomicOr(p.status, kStatusBadPage);
        id = 0;
      }
      if (lane < 8) sh.ids[at][lane] = has ? id : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.g_full[at]);
      sc = 1.f;
      if (has) sc = p.scales[id];
      advance(look);
      id = fetch();
      ++lg;
    };
    look_up();
    int slot = 2, issued = 0;
    uint32_t ph = 1;
    for (int g = 0; !c.done; ++g) {
      if (c.j == 0) n = tokens(c);
      const int valid = min(CT, n - (c.s.c0 + c.j) * CT);
      const int blocks = (valid + p.bs - 1) >> p.lbs;
      bool ok = true;
#pragma unroll 1
      for (int a = 2; a < 4; ++a) {
        ok = warp_wait(&sh.c_empty[slot], ph, abort_v, p.status);
        if (!ok) break;
        if (elect_one()) load_box(a, slot, blocks, sh.ids[g % GR]);
        issued = 4 * g + a + 1;
        __syncwarp();
        slot += a == 2 ? 1 : 3;
        if (slot >= NS) { slot -= NS; ph ^= 1; }
      }
      if (!ok) break;
      while (lg <= g + AHEAD && (pending || !look.done)) look_up();
      advance(c);
    }
    if (lane == 0) sh.issued[1] = issued;
  } else {
    // ---------------- softmax: thread = token, group = HPG heads
    const int grp = (warp - 4) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const int h0 = grp * HPG, bar = 1 + grp;
    const int tg = (int)threadIdx.x - 128 - 128 * grp;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t p_base = smem_u32(smem + K::OFF_P);
    const int head0 = hg * p.hg_heads + h0;   // this group's first head
    const int n_heads = max(0, min(min(HPG, p.hg_heads - h0), p.h - head0));   // real ones
    float* const inv_w = sh.inv[grp][quad];   // this warp's 2^-k per head
    bool ok = true;
    int g = 0;
    for (; !c.done; c.next_seg(p.pre, p.B, sl, u)) {
      const Seg s = c.s;
      const int n = tokens(c);
      if (tg < HPG) {
        sh.hf[h0 + tg] = p.qf[((int64_t)s.b * p.groups + hg) * NH + h0 + tg];
        sh.nref[h0 + tg] = 0.f;               // the first chunk sets it
      }
      named_barrier_sync(bar, 128);
      float l[HPG];
#pragma unroll
      for (int i = 0; i < HPG; ++i) l[i] = 0.f;
      for (int j = 0; j < s.nch; ++j, ++g) {
        const int sls = g % NSL, pb = g % NP;
        const bool live = row < n - (s.c0 + j) * CT;
        ok = ok && warp_wait(&sh.e_full[g % GR], (g / GR) & 1, abort_v, p.status);
        const float sc = sh.scl[g % GR][row >> p.lbs];
        ok = ok && warp_wait(&sh.s_full[sls], (g / NSL) & 1, abort_v, p.status);
        float v[HPG], vm = -INFINITY;
        {
          uint32_t a[HPG], b[HPG];
          tc_fence_after();
          const uint32_t ts = tbase + lane_off + K::TM_S + sls * 2 * NH + h0;
          tmem_ld_n<HPG>(ts, a);
          tmem_ld_n<HPG>(ts + NH, b);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.s_free[sls]);
          // v = raw 2^e f - ref
#pragma unroll
          for (int i = 0; i < HPG; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sh.hf[h0 + i]);
            const float4 r = *reinterpret_cast<const float4*>(&sh.nref[h0 + i]);
            const float ff[4] = {f.x, f.y, f.z, f.w}, rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              float x = __uint_as_float(a[i + k]), y = __uint_as_float(a[i + k + 1]);
              add2(x, y, __uint_as_float(b[i + k]), __uint_as_float(b[i + k + 1]));
              mul2(x, y, sc, sc);
              fma2(v[i + k], v[i + k + 1], x, y, ff[k], ff[k + 1], rr[k], rr[k + 1]);
              vm = max3f(vm, v[i + k], v[i + k + 1]);
            }
          }
        }
        if (!live) {                          // behind the last token
#pragma unroll
          for (int i = 0; i < HPG; ++i) v[i] = -INFINITY;
        }
        if (j == 0) {
          // the first token's scores are the segment's first references (nref
          // may still be read as 0 by a slower warp before the barrier)
          if (row == 0) {
#pragma unroll
            for (int i = 0; i < HPG; ++i) sh.alpha[h0 + i] = -v[i];
          }
          named_barrier_sync(bar, 128);
          if (tg < HPG) sh.nref[h0 + tg] = sh.alpha[h0 + tg];
          vm = -INFINITY;
#pragma unroll
          for (int i = 0; i < HPG; ++i) {
            v[i] += sh.alpha[h0 + i];
            vm = fmaxf(vm, v[i]);
          }
        }
        // the rare case: a score far above its reference (or a warp that gave up)
        const bool far = barrier_or(bar, 128, !ok || (live && vm > kGrow));
        if (far) {
          // new references; if a warp gave up, the group leaves together
          if (barrier_or(bar, 128, !ok)) { ok = false; break; }
          int mine = 0;
#pragma unroll
          for (int i = 0; i < HPG; ++i) {
            v[i] -= sh.nref[h0 + i];          // the score itself
            const int k = __reduce_max_sync(0xffffffffu, float_key(v[i]));
            if (lane == i) mine = k;
          }
          if (lane < HPG) sh.hmax[grp][quad][lane] = mine;
          named_barrier_sync(bar, 128);
          if (quad == 0 && lane < HPG) {
            const float x = key_float(max(max(sh.hmax[grp][0][lane], sh.hmax[grp][1][lane]),
                                          max(sh.hmax[grp][2][lane], sh.hmax[grp][3][lane])));
            const float old = -sh.nref[h0 + lane], now = x > old ? x : old;
            sh.nref[h0 + lane] = -now;
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
          for (int i = 0; i < HPG; ++i) v[i] += sh.nref[h0 + i];
        }
        // p, its row sums, and p 2^e
        uint32_t m[HPG / 2];
#pragma unroll
        for (int i = 0; i < HPG; i += 2) {
          v[i] = ex2(v[i]);
          v[i + 1] = ex2(v[i + 1]);
          add2(l[i], l[i + 1], v[i], v[i + 1]);
          mul2(v[i], v[i + 1], sc, sc);
          m[i / 2] = __byte_perm(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), 0x7632);
        }
        // The largest of the warp's 32 tokens per head, from the upper halves of
        // the (non-negative) floats, whose order is that of their bits, NaN above
        // all: lanes trade halves of their heads until a lane has two.  (A
        // redux.sync per head, 16 one after the other, took 8 % longer.)
        int pair = 0;
#pragma unroll
        for (int w = HPG / 4, o = 16; o; w >>= 1, o >>= 1) {
          if (w > 0) {
            const bool up = lane & o;
            pair = 2 * pair + up;
#pragma unroll
            for (int i = 0; i < w; ++i) {
              const uint32_t give = up ? m[i] : m[i + w], mine = up ? m[i + w] : m[i];
              m[i] = max_u16x2(mine, __shfl_xor_sync(0xffffffffu, give, o));
            }
          } else {
            m[0] = max_u16x2(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
          }
        }
        // it goes to [128, 256): factor 2^-k, and the scale 2^k as a ue8m0 byte
        const uint32_t ex0 = max(m[0] & 0x7f80u, 8u << 7) << 16;
        const uint32_t ex1 = max((m[0] >> 16) & 0x7f80u, 8u << 7) << 16;
        constexpr int SAME = 64 / HPG;        // lanes with the same pair
        if (lane % SAME == 0)
          *reinterpret_cast<float2*>(inv_w + 2 * pair) =
              make_float2(__uint_as_float(0x82800000u - ex0), __uint_as_float(0x82800000u - ex1));
        __syncwarp();
        uint32_t hb[HPG / 4], lb[HPG / 4];
#pragma unroll
        for (int i = 0; i < HPG / 4; ++i) {
          const float4 f = *reinterpret_cast<const float4*>(inv_w + 4 * i);
          float* const w = v + 4 * i;
          mul2(w[0], w[1], f.x, f.y);
          mul2(w[2], w[3], f.z, f.w);
          const uint32_t w01 = pack_f16(w[0], w[1]), w23 = pack_f16(w[2], w[3]);
          const uint32_t h01 = f16x2_to_e4m3x2(w01), h23 = f16x2_to_e4m3x2(w23);
          hb[i] = h01 | (h23 << 16);
          lb[i] = f16x2_to_e4m3x2(sub_f16x2(w01, e4m3x2_to_f16x2(h01))) |
                  (f16x2_to_e4m3x2(sub_f16x2(w23, e4m3x2_to_f16x2(h23))) << 16);
        }
        // PV of chunk g - NP has run: this P buffer and its scales are free
        if (g >= NP) ok = ok && warp_wait(&sh.pv_done[pb], ((g / NP) - 1) & 1, abort_v, p.status);
        if (lane % SAME == 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int nh = h0 + 2 * pair + k;
            const uint8_t sfb = (uint8_t)(((k ? ex1 : ex0) >> 23) - 7);
            sh.sf[pb][(nh & 31) * 16 + (nh >> 5) * 4 + quad] = sfb;
            if (K::STK) sh.sf[pb][((nh + NH) & 31) * 16 + ((nh + NH) >> 5) * 4 + quad] = sfb;
          }
        }
        const uint32_t pt = p_base + pb * K::PBYTES;
        constexpr uint32_t lo_at = K::STK ? NH : 0, lo_tile = K::STK ? 0 : CT * 64;
        const uint32_t at = row * K::PW + h0;
        if constexpr (HPG == 16) {
          st_shared_v4(pt + swz<K::PW>(at), hb[0], hb[1], hb[2], hb[3]);
          st_shared_v4(pt + lo_tile + swz<K::PW>(at + lo_at), lb[0], lb[1], lb[2], lb[3]);
        } else {
          st_shared_v2(pt + swz<K::PW>(at), hb[0], hb[1]);
          st_shared_v2(pt + lo_tile + swz<K::PW>(at + lo_at), lb[0], lb[1]);
        }
        // a weight of 0 times whatever lies behind the last token could be NaN
        // (neighbouring rows take their pieces in another order: one bank's
        // would make it 2 us for a chunk of a few tokens)
        if (!live) {
          for (int i = grp; i < 32; i += NG) {
            const int slot = (4 * g + (i >> 3)) % NS;
            st_shared_v4(smem_u32(smem + K::OFF_C + slot * BOX) + row * 128 +
                             (((i + lane) & 7) << 4), 0, 0, 0, 0);
          }
        }
        fence_proxy_async();
        tc_fence_before();                    // a rescaled O comes before this PV
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[pb]);
      }
      // Segment end: row sums over the 128 tokens, then the output
      if (barrier_or(bar, 128, !ok)) break;
      {
        // lanes trade halves of their heads until a lane has one
        int head = 0;
#pragma unroll
        for (int w = HPG / 2, o = 16; o; w >>= 1, o >>= 1) {
          if (w > 0) {
            const bool up = lane & o;
            head = 2 * head + up;
#pragma unroll
            for (int i = 0; i < w; ++i) {
              const float give = up ? l[i] : l[i + w], mine = up ? l[i + w] : l[i];
              l[i] = mine + __shfl_xor_sync(0xffffffffu, give, o);
            }
          } else {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
          }
        }
        if (lane % (32 / HPG) == 0) sh.lsum[grp][quad][head] = l[0];
      }
      named_barrier_sync(bar, 128);
      if (lane < HPG) {
        const float sum = (sh.lsum[grp][0][lane] + sh.lsum[grp][1][lane]) +
                          (sh.lsum[grp][2][lane] + sh.lsum[grp][3][lane]);
        sh.alpha[h0 + lane] = 1.f / sum;        // the same from all four warps
        if (!s.whole && quad == 0 && lane < n_heads)
          p.part_lse[(int64_t)s.slot * p.h + head0 + lane] = log2f(sum) - sh.nref[h0 + lane];
      }
      __syncwarp();
      ok = warp_wait(&sh.o_done, c.kk & 1, abort_v, p.status);
      tc_fence_after();
      if (ok) {
        float inv[HPG];
#pragma unroll
        for (int k = 0; k < HPG; ++k) inv[k] = sh.alpha[h0 + k];
#pragma unroll 1
        for (int a = 0; a < 4; ++a) {
          uint32_t o[HPG], o2[HPG];
          const uint32_t to = tbase + lane_off + K::TM_O + a * K::PN + h0;
          tmem_ld_n<HPG>(to, o);
          if (K::STK) tmem_ld_n<HPG>(to + NH, o2);
          tmem_wait_ld();
          if (a == 3) {
            tc_fence_before();                // O may be overwritten
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.o_free);
          }
          const int dim = a * 128 + row;
          float* dst = (s.whole ? p.o_lat + ((int64_t)s.b * p.h + head0) * R
                                : p.part_o + ((int64_t)s.slot * p.h + head0) * R) + dim;
#pragma unroll
          for (int k = 0; k < HPG; ++k) {
            float x = __uint_as_float(o[k]);
            if (K::STK) x += __uint_as_float(o2[k]);
            if (k < n_heads) dst[k * R] = x * inv[k];
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_v) drain<NH>(sh);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, K::TM_COLS);
  }
}

template <int NH>
cudaError_t launch_attn(const AttnParams& p, const CUtensorMap& tmQ, const CUtensorMap& tmQr,
                        const CUtensorMap& tmC, const CUtensorMap& tmCr, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_attn_kernel<NH>, smem_bytes<NH>(), set);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_attn_kernel<NH>, dim3(p.n_units * p.groups), dim3(Cfg<NH>::NTHREADS),
                    smem_bytes<NH>(), st, tmQ, tmQr, tmC, tmCr, p);
}

}  // namespace

bool tc_paged_supported(const mla_config& c) { return tc_decode_supported(c); }

PagedTcPlan tc_paged_plan(int h, int sms) {
  PagedTcPlan t;
  t.groups = (h + 63) / 64;
  t.hg_heads = (h + t.groups - 1) / t.groups;
  t.NH = (t.hg_heads + 15) / 16 * 16;
  const int n = sms / t.groups;
  t.n_units = n < 1 ? 1 : n > 512 ? 512 : n;   // 512: what the output kernel merges
  return t;
}

cudaError_t tc_paged_decode(const PagedDecodeArgs& a, cudaStream_t st) {
  const PagedTcPlan& t = a.tc;
  constexpr int kMinLen = 1;                // shortest slice, chunks
  cudaError_t e = launch_paged_query(a, kMinLen, st);
  if (e != cudaSuccess) return e;
  stage_event(1, st);
  // e4m3 tensors as pairs of bytes: 288 columns of 16 bits
  CUtensorMap tmQ, tmQr, tmC, tmCr;
  const uint64_t str[1] = {(uint64_t)W};
  const uint64_t qdims[2] = {W / 2, (uint64_t)a.B * t.groups * 2 * t.NH};
  const uint32_t qbox[2] = {64, (uint32_t)(2 * t.NH)}, qrbox[2] = {DR / 2, (uint32_t)(2 * t.NH)};
  const uint64_t cdims[2] = {W / 2, (uint64_t)a.pool.n_blocks * a.pool.bs};
  const uint32_t cbox[2] = {64, (uint32_t)a.pool.bs}, crbox[2] = {DR / 2, (uint32_t)a.pool.bs};
  if (!encode_tmap(&tmQ, a.q8, 2, qdims, str, qbox) ||
      !encode_tmap(&tmQr, a.q8, 2, qdims, str, qrbox, 64) ||
      !encode_tmap(&tmC, a.pool.cache, 2, cdims, str, cbox) ||
      !encode_tmap(&tmCr, a.pool.cache, 2, cdims, str, crbox, 64))
    return cudaErrorInvalidValue;
  AttnParams p{};
  p.pre = a.pre; p.len = a.len; p.first = (const int4*)a.first; p.table = a.table;
  p.scales = a.pool.scales; p.qf = a.qf;
  p.B = a.B; p.max_blocks = a.max_blocks; p.n_blocks = a.pool.n_blocks; p.bs = a.pool.bs;
  p.lbs = a.pool.bs == 16 ? 4 : a.pool.bs == 32 ? 5 : a.pool.bs == 64 ? 6 : 7;
  p.h = a.h; p.groups = t.groups; p.hg_heads = t.hg_heads;
  p.n_units = t.n_units; p.min_len = kMinLen;
  p.part_o = a.part_o; p.part_lse = a.part_lse;
  p.o_lat = (float*)a.o_lat;
  p.status = a.status;
  e = t.NH == 16   ? launch_attn<16>(p, tmQ, tmQr, tmC, tmCr, st)
      : t.NH == 32 ? launch_attn<32>(p, tmQ, tmQr, tmC, tmCr, st)
      : t.NH == 48 ? launch_attn<48>(p, tmQ, tmQr, tmC, tmCr, st)
                   : launch_attn<64>(p, tmQ, tmQr, tmC, tmCr, st);
  count_launches();
  if (e != cudaSuccess) return e;
  stage_event(2, st);
  e = launch_paged_output(a, st);
  if (e != cudaSuccess) return e;
  stage_event(3, st);
  return cudaGetLastError();
}

}  // namespace mla
