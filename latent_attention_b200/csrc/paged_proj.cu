// The two projections around the tensor-core paged attention, one head and up
// to 128 sequences a block:
//
//   paged_query_kernel   q_lat = W_UK[h]^T q_nope, and [q_lat | q_pe] as two
//                        e4m3 terms and a power of two; the lengths and the
//                        chunk line of all sequences
//   paged_output_kernel  o_lat of every sequence from its partial results, and
//                        o = W_UV[h] o_lat
//
// Both read each head's 128 KB of weights once and do little with them (a
// decode batch has tens of rows): what bounds them is the time of a launch, of
// one trip to memory and of fetching their instructions, so the work around
// the products (rounding to 8 bits, merging) is done where the operands are.
// The query's product is warp-level MMAs, whose results the threads round where
// they hold them, a row of q_lat in one warp's quads; the output's is tcgen05
// with the 128 columns as M and the sequences as N (as warp-level MMAs, some 19
// cycles each, it took 5000 cycles of 12500 for 16 sequences).  (Four blocks a
// head, in a cluster, took longer: 45 us against 26 for both kernels at 64
// sequences of 128 heads.)  Neither q_lat nor o_lat is rounded to 16 bits: q_lat
// goes from fp32 to its two terms, o_lat enters the product as two bf16 terms (16
// significant bits).  A whole call of 4 sequences and 128 heads takes 23.1 us, of
// which the two kernels take some 6 each: the 33 MB of weights would take 5.
#include <algorithm>

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
constexpr int NT = 512;                  // threads, 16 warps
constexpr int MB = 32;                   // sequences in a round

// Rounds a block: one while the blocks have SMs of their own (the weights are
// then read by several), more beyond, up to four.
int rounds_of(const PagedDecodeArgs& a) {
  const int64_t blocks = (int64_t)a.h * ((a.B + MB - 1) / MB);
  return (int)std::min<int64_t>(4, (blocks + kSMs - 1) / kSMs);
}
constexpr int WBOX = 128 * 128;          // 128 rows of 64 bf16 weights
constexpr int W_BYTES = 8 * WBOX;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte column c of row r in a box of 128-byte rows, 128-byte
// swizzle.
__device__ __forceinline__ uint32_t box_at(int r, int c) {
  return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

// ------------------------------------------------------------------- query
struct QueryParams {
  const __nv_bfloat16 *q_nope, *q_pe;      // [B, h, dn], [B, h, DR]
  uint8_t* q8;                             // [B, groups, 2, NH, W]
  float* qf;                               // [B, groups, NH]
  const int32_t* ctx;
  int64_t* pre;
  int32_t *len, *first;
  int2* parts;
  int B, h, dn, dv, groups, hg_heads, NH, n_units, min_len, rounds;
  int64_t most;                            // tokens a table holds
  float scale_log2;
  uint32_t* status;
};
constexpr int Q_TILE = MB * 256;           // 32 rows of 128 bf16, two boxes of 64 columns
constexpr int Q_SMEM = W_BYTES + Q_TILE + 1024;

// Two e4m3 terms of a pair: hi in the low half, lo in the high half.
__device__ __forceinline__ uint32_t split_pair(float x, float y) {
  const uint32_t hi = to_e4m3x2(x, y);
  float b[2];
  {
    float t[4];
    from_e4m3x4(hi, t);
    b[0] = t[0]; b[1] = t[1];
  }
  return hi | (to_e4m3x2(x - b[0], y - b[1]) << 16);
}
// |x| as bits for the row's maximum; an infinity becomes NaN (e4m3 has none)
// and, like NaN, does not set the scale.
__device__ __forceinline__ uint32_t finite_bits(float& x) {
  const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
  if (a < 0x7f800000u) return a;
  x = x - x;
  return 0;
}

__device__ void lengths(const QueryParams& p) {
  __shared__ int64_t sums[NT / 32];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) p.status[0] = p.status[1] = 0;
  __syncthreads();
  const int per = (p.B + NT - 1) / NT, b0 = min(t * per, p.B), b1 = min(b0 + per, p.B);
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
  __syncthreads();
  // every sequence's partial results: the slot of the first, their number (1:
  // the whole sequence, not in a slot; 0: no tokens).  The others' slots are
  // those of the next units' first segments.
  for (int b = t; b < p.B; b += NT) {
    int2 x = make_int2(0, 0);
    if (p.len[b] > 0) {
      const SeqUnits su = seq_units(p.pre, b, p.B, p.n_units, p.min_len);
      x = make_int2(seq_slot(su, su.u0), su.u1 - su.u0 + 1);
    }
    p.parts[b] = x;
  }
  // every unit's first segment: the attention kernel starts with one load
  for (int u = t; u < p.n_units; u += NT) {
    const Slice sl = unit_slice(p.pre, p.B, u, p.n_units, p.min_len);
    Cursor c;
    c.start(p.pre, p.B, sl, u, seq_at(p.pre, p.B, sl.r0));
    int4* rec = reinterpret_cast<int4*>(p.first) + 2 * u;
    const Seg& s = c.s;
    rec[0] = c.done ? make_int4(0, 0, 0, 0) : make_int4(s.b, s.c0, s.nch, s.slot);
    rec[1] = c.done ? make_int4(0, 0, 0, 0) : make_int4(s.whole, p.len[s.b], 0, 0);
  }
}

// The 16-bit values that the four lanes of a quad hold of each of four groups
// (v[n]: group n), handed over so that a lane ends with group (lane & 3), in the
// lanes' order.
__device__ __forceinline__ uint2 quad_transpose(const uint32_t (&v)[4], int lane) {
  const uint32_t a = __byte_perm(v[0], v[1], 0x5410), b = __byte_perm(v[2], v[3], 0x5410);
  const bool up = lane & 2, odd = lane & 1;
  const uint32_t k = up ? b : a, o = __shfl_xor_sync(0xffffffffu, up ? a : b, 2);
  const uint32_t lo = __byte_perm(k, o, 0x5410), hi = __byte_perm(k, o, 0x7632);
  // (this lane, lane ^ 2) and (lane ^ 1, lane ^ 3) of this lane's group
  const uint32_t x = odd ? hi : lo, y = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
  const uint32_t e = odd ? y : x, f = odd ? x : y;
  const uint32_t w0 = __byte_perm(e, f, 0x5410), w1 = __byte_perm(e, f, 0x7632);
  return up ? make_uint2(w1, w0) : make_uint2(w0, w1);
}

// Block (x, y): x = 0 the lengths, 1 .. h a head, from h + 1 on a row that pads
// the head groups (a block each: one block for 15 of them took 12 us longer); y:
// 32 x rounds sequences
__global__ void __launch_bounds__(NT) paged_query_kernel(const __grid_constant__ CUtensorMap tmW,
                                                         QueryParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full;
  __shared__ int abort_flag;
  __shared__ uint32_t amax_s[2][MB];       // the rows' maxima, of even and odd rounds
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    mbar_init(&full, 1);
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tmW);
  }
  if (t < 2 * MB) amax_s[t / MB][t % MB] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int b0 = blockIdx.y * MB * p.rounds, nb = min(MB * p.rounds, p.B - b0);
  if (blockIdx.x == 0) {
    if (blockIdx.y == 0) lengths(p);
    return;
  }
  if ((int)blockIdx.x > p.h) {
    // pad row j: groups are full but for the last rows of each
    int g = 0, i = (int)blockIdx.x - p.h - 1;
    for (; g < p.groups; ++g) {
      const int real = min(p.hg_heads, p.h - g * p.hg_heads), n = p.NH - real;
      if (i < n) { i += real; break; }
      i -= n;
    }
    for (int k = t; k < nb * 2 * (W / 16); k += NT) {
      const int c = k % (W / 16), term = k / (W / 16) % 2;
      const int64_t bg = (int64_t)(b0 + k / (W / 8)) * p.groups + g;
      *reinterpret_cast<uint4*>(p.q8 + ((bg * 2 + term) * p.NH + i) * W + c * 16) =
          make_uint4(0u, 0u, 0u, 0u);
      if (c == 0 && term == 0) p.qf[bg * p.NH + i] = 0.f;
    }
    return;
  }
  const int hh = blockIdx.x - 1;
  const int g = hh / p.hg_heads, i = hh % p.hg_heads;
  const uint32_t wbase = smem_u32(smem), qbase = wbase + W_BYTES;
  const int r = lane >> 2;
  // a 16-byte piece of q_nope and four values of q_pe a thread
  const int rr = t >> 4, part = t & 15;
  int phase = 0;
  for (int round = 0; round * MB < nb; ++round) {
    const int base = b0 + round * MB, n = min(MB, nb - round * MB);
    float acc[2][4][4];                    // 32 rows x this warp's 32 dims
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[m][q][k] = 0.f;
    uint2 pe2 = make_uint2(0u, 0u);
    if (rr < n)
      pe2 = reinterpret_cast<const uint2*>(p.q_pe + ((int64_t)(base + rr) * p.h + hh) * DR)[part];
    for (int kc = 0; kc < p.dn; kc += 128) {
      // 128 rows of W_UK[h]; past dn they are W_UV's and the next head's, and
      // become zeros (to meet zeros of q is not enough for an infinity or NaN).
      // Up to 128 rows they stay for all rounds.
      const bool load = round == 0 || p.dn > 128;
      if (t == 0 && load) {
        mbar_arrive_expect_tx(&full, W_BYTES);
        for (int x = 0; x < 8; ++x)
          tma_load_2d(smem + x * WBOX, &tmW, 64 * x, hh * (p.dn + p.dv) + kc, &full);
      }
      uint4 q4 = make_uint4(0u, 0u, 0u, 0u);
      if (rr < n && kc + 8 * part < p.dn)
        q4 = *reinterpret_cast<const uint4*>(p.q_nope + ((int64_t)(base + rr) * p.h + hh) * p.dn +
                                             kc + 8 * part);
      st_shared_v4(qbase + (part >> 3) * (Q_TILE / 2) + box_at(rr, part & 7), q4.x, q4.y, q4.z,
                   q4.w);
      __syncthreads();
      // (after a timeout the block goes on; the status word says so)
      if (load) {
        mbar_wait(&full, phase++ & 1, &abort_flag, p.status);
        const int past = kc + 128 - p.dn;
        if (past > 0) {
          for (int k = t; k < 64 * past; k += NT)
            st_shared_v4(wbase + (k & 7) * WBOX + (127 - (k >> 6)) * 128 + ((k >> 3) & 7) * 16, 0u,
                         0u, 0u, 0u);
          fence_proxy_async();             // before the loads that come into their place
          __syncthreads();
        }
      }
#pragma unroll 2
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t a[2][4], b[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (m == 0 || n > 16)
            ldsm4(qbase + (ks >> 2) * (Q_TILE / 2) +
                      box_at(m * 16 + (lane & 15), 2 * (ks & 3) + (lane >> 4)), a[m]);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          ldsm4_t(wbase + (warp >> 1) * WBOX +
                      box_at(ks * 16 + (lane & 15), 4 * (warp & 1) + 2 * q + (lane >> 4)), b[q]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m == 1 && n <= 16) continue;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            mma16816(acc[m][2 * q], a[m], b[q][0], b[q][1]);
            mma16816(acc[m][2 * q + 1], a[m], b[q][2], b[q][3]);
          }
        }
      }
      __syncthreads();                     // weights and q are read
    }
    // the rows' maxima
    uint32_t* amax = amax_s[round & 1];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m == 1 && n <= 16) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t y = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          y = max(y, max(finite_bits(acc[m][q][2 * half]), finite_bits(acc[m][q][2 * half + 1])));
        y = max(y, __shfl_xor_sync(0xffffffffu, y, 1));
        y = max(y, __shfl_xor_sync(0xffffffffu, y, 2));
        if ((lane & 3) == 0) atomicMax(&amax[m * 16 + half * 8 + r], y);
      }
    }
    float pe[4] = {__uint_as_float(pe2.x << 16), __uint_as_float(pe2.x & 0xffff0000u),
                   __uint_as_float(pe2.y << 16), __uint_as_float(pe2.y & 0xffff0000u)};
    {
      uint32_t y = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) y = max(y, finite_bits(pe[k]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) y = max(y, __shfl_xor_sync(0xffffffffu, y, o));
      if (part == 0) atomicMax(&amax[rr], y);
    }
    __syncthreads();
    if (t < MB) amax_s[~round & 1][t] = 0;  // for the next round (its barriers lie between)
#pragma unroll 1
    for (int mh = 0; mh < (n > 16 ? 4 : 2); ++mh) {
      const int row = (mh >> 1) * 16 + (mh & 1) * 8 + r;
      const float f = pow2(-scale_exp(amax[row]));
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x, y;
        x = mh == 0 ? acc[0][q][0] : mh == 1 ? acc[0][q][2] : mh == 2 ? acc[1][q][0] : acc[1][q][2];
        y = mh == 0 ? acc[0][q][1] : mh == 1 ? acc[0][q][3] : mh == 2 ? acc[1][q][1] : acc[1][q][3];
        const uint32_t v = split_pair(x * f, y * f);
        hi[q] = v & 0xffffu;
        lo[q] = v >> 16;
      }
      const uint2 h2 = quad_transpose(hi, lane), l2 = quad_transpose(lo, lane);
      if (row < n) {
        uint8_t* dst = p.q8 + (((int64_t)(base + row) * p.groups + g) * 2 * p.NH + i) * W +
                       warp * 32 + 8 * (lane & 3);
        *reinterpret_cast<uint2*>(dst) = h2;
        *reinterpret_cast<uint2*>(dst + (int64_t)p.NH * W) = l2;
      }
    }
    if (rr < n) {
      const int e = scale_exp(amax[rr]);
      const float f = pow2(-e);
      const uint32_t v0 = split_pair(pe[0] * f, pe[1] * f), v1 = split_pair(pe[2] * f, pe[3] * f);
      const int64_t bg = (int64_t)(base + rr) * p.groups + g;
      uint8_t* dst = p.q8 + (bg * 2 * p.NH + i) * W + R + 4 * part;
      *reinterpret_cast<uint32_t*>(dst) = __byte_perm(v0, v1, 0x5410);
      *reinterpret_cast<uint32_t*>(dst + (int64_t)p.NH * W) = __byte_perm(v0, v1, 0x7632);
      if (part == 0) p.qf[bg * p.NH + i] = p.scale_log2 * pow2(e);
    }
  }
}

// ------------------------------------------------------------------ output
struct OutputParams {
  const float *part_o, *part_lse;          // [2 n_units, h, R], [2 n_units, h] (log2)
  const float* o_lat;                      // [B, h, R]: sequences in one segment
  const int2* parts;                       // [B] slot of the first partial, their number
  __nv_bfloat16 *out, *out_lo;             // [B, h, dv]; what is left of it, or null
  int B, h, dn, dv, rounds;
  uint32_t* status;
};
constexpr int A_BYTES = 8 * MB * 128;      // o_lat of 32 sequences, one bf16 term
constexpr int RED = 8 * R * 4;             // the merge of many partials
constexpr int O_SMEM = W_BYTES + 2 * A_BYTES + RED + 1024;
constexpr int kUnits = 512;                // most units (host side: tc_paged_plan)
constexpr int kShared = 8;                 // more partials than this: the whole block merges

__global__ void __launch_bounds__(NT) paged_output_kernel(const __grid_constant__ CUtensorMap tmW,
                                                          OutputParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full, done;
  __shared__ int abort_flag;
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t many;                // rows that the whole block merges
  __shared__ const float* src_s[MB][kShared];   // a row's partials
  __shared__ float w_s[MB][kShared];       // and their weights
  __shared__ float u_s[2 * kUnits];        // lse and weights of one row with many partials
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int hh = blockIdx.x;
  const int b0 = blockIdx.y * MB * p.rounds, nb = min(MB * p.rounds, p.B - b0);
  const uint32_t wbase = smem_u32(smem), abase = wbase + W_BYTES;
  float* red = reinterpret_cast<float*>(smem + W_BYTES + 2 * A_BYTES);
  auto load_w = [&](int nc) {
    mbar_arrive_expect_tx(&full, W_BYTES);
    for (int i = 0; i < 8; ++i)
      tma_load_2d(smem + i * WBOX, &tmW, 64 * i, hh * (p.dn + p.dv) + p.dn + nc, &full);
  };
  if (t == 0) {
    mbar_init(&full, 1);
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_barrier_init();
    // The weights do not depend on the kernel before this one (which started
    // only once all before it had finished): they are on their way while it
    // ends.
    load_w(0);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, 32);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base;
  griddep_wait();
  griddep_launch_dependents();

  // four dims of a row as two bf16 terms into the B operand's boxes
  auto put = [&](int row, int d, const float4& v) {
    const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
    const uint32_t l0 = pack_bf16(v.x - __uint_as_float(h0 << 16),
                                  v.y - __uint_as_float(h0 & 0xffff0000u));
    const uint32_t l1 = pack_bf16(v.z - __uint_as_float(h1 << 16),
                                  v.w - __uint_as_float(h1 & 0xffff0000u));
    uint8_t* at = smem + W_BYTES + (d >> 6) * MB * 128 + box_at(row, (d & 63) >> 3) + (d & 7) * 2;
    *reinterpret_cast<uint2*>(at) = make_uint2(h0, h1);
    *reinterpret_cast<uint2*>(at + A_BYTES) = make_uint2(l0, l1);
  };
  // slot of partial i of a sequence
  auto slot_of = [](const int2& x, int i) { return i == 0 ? x.x : 2 * ((x.x >> 1) + i); };
  int phase = 0, runs = 0;
  bool coming = true;                      // weights are on their way
  for (int round = 0; round * MB < nb; ++round) {
    const int base = b0 + round * MB, n = min(MB, nb - round * MB);
    const int rows = n <= 16 ? 16 : 32;    // N of the product
    if (t == 0) many = 0;
    __syncthreads();
    // a thread per row and partial: where it lies, and its weight
    if (t < MB * kShared) {
      const int row = t / kShared, i = t % kShared, b = base + row;
      const int2 x = row < n ? p.parts[b] : make_int2(0, 0);
      const float* src = nullptr;
      float w = 1.f;
      if (x.y == 1) {
        if (i == 0) src = p.o_lat + ((int64_t)b * p.h + hh) * R;
      } else if (x.y > kShared) {
        if (i == 0) atomicOr(&many, 1u << row);
      } else if (i < x.y) {
        const int64_t at = (int64_t)slot_of(x, i) * p.h + hh;
        src = p.part_o + at * R;
        w = p.part_lse[at];
      }
      // (eight neighbouring lanes hold a row)
      const bool part = x.y > 1 && x.y <= kShared && i < x.y;
      float mx = part ? w : -INFINITY;
#pragma unroll
      for (int o = 1; o < kShared; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (part) w = exp2f(w - mx);
      float den = part ? w : 0.f;
#pragma unroll
      for (int o = 1; o < kShared; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      src_s[row][i] = src;
      w_s[row][i] = part ? w / den : 1.f;
    }
    __syncthreads();
#pragma unroll 1
    for (int row = warp; row < rows; row += NT / 32) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      // two partials (32 bytes a lane and 128 dims) in flight
#pragma unroll 1
      for (int i = 0; i < kShared && src_s[row][i]; i += 2) {
        const float *s0 = src_s[row][i], *s1 = src_s[row][i + 1];
        const float w0 = w_s[row][i], w1 = w_s[row][i + 1];
        float4 x[4], y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = reinterpret_cast<const float4*>(s0)[lane + 32 * q];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          y[q] = s1 ? reinterpret_cast<const float4*>(s1)[lane + 32 * q]
                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[q].x = fmaf(w1, y[q].x, fmaf(w0, x[q].x, v[q].x));
          v[q].y = fmaf(w1, y[q].y, fmaf(w0, x[q].y, v[q].y));
          v[q].z = fmaf(w1, y[q].z, fmaf(w0, x[q].z, v[q].z));
          v[q].w = fmaf(w1, y[q].w, fmaf(w0, x[q].w, v[q].w));
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) put(row, 4 * lane + 128 * q, v[q]);
    }
    for (uint32_t left = many; left; left &= left - 1) {
      const int row = __ffs(left) - 1;
      const int2 x = p.parts[base + row];  // (at most kUnits partials)
      float mx = -INFINITY, den = 0.f;
      __syncthreads();
      for (int i = t; i < x.y; i += NT) u_s[i] = p.part_lse[(int64_t)slot_of(x, i) * p.h + hh];
      __syncthreads();
      for (int i = lane; i < x.y; i += 32) mx = fmaxf(mx, u_s[i]);
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      for (int i = t; i < x.y; i += NT) u_s[kUnits + i] = exp2f(u_s[i] - mx);
      __syncthreads();
      // every eighth partial and half of the dims a warp
      float4 v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int at = lane + 64 * (warp >> 3);
#pragma unroll 4
      for (int i = warp & 7; i < x.y; i += 8) {
        const float4* src =
            reinterpret_cast<const float4*>(p.part_o + ((int64_t)slot_of(x, i) * p.h + hh) * R);
        const float w = u_s[kUnits + i];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 y = src[at + 32 * q];
          v[q].x = fmaf(w, y.x, v[q].x); v[q].y = fmaf(w, y.y, v[q].y);
          v[q].z = fmaf(w, y.z, v[q].z); v[q].w = fmaf(w, y.w, v[q].w);
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q)
        reinterpret_cast<float4*>(red + (warp & 7) * R)[at + 32 * q] = v[q];
      for (int i = lane; i < x.y; i += 32) den += u_s[kUnits + i];
#pragma unroll
      for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      __syncthreads();
      if (t < R / 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < 8; ++w) {
          const float4 z = reinterpret_cast<const float4*>(red + w * R)[t];
          y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        }
        const float inv = 1.f / den;
        y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
        put(row, 4 * t, y);
      }
    }
    fence_proxy_async();                   // the operand's boxes, to the tensor core
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // up to 128 output columns the weights stay for all rounds
    for (int nc = 0; nc < p.dv; nc += 128) {
      if (!coming && p.dv > 128) {
        if (t == 0) load_w(nc);
        coming = true;
      }
      // (after a timeout the block goes on; the status word says so)
      if (coming) mbar_wait(&full, phase++ & 1, &abort_flag, p.status);
      coming = false;
      // the columns as M, the sequences as N
      if (warp == 0 && elect_one()) {
        const uint32_t idesc = idesc_bf16(128, rows);
#pragma unroll 1
        for (int box = 0; box < 8; ++box) {
          const uint64_t da = desc_kmajor_sw128(wbase + box * WBOX);
          const uint64_t dh = desc_kmajor_sw128(abase + box * MB * 128);
          const uint64_t dl = desc_kmajor_sw128(abase + A_BYTES + box * MB * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mma_bf16_keep<false>(tbase, da + 2 * k, dh + 2 * k, idesc, (box | k) != 0);
            mma_bf16_keep<true>(tbase, da + 2 * k, dl + 2 * k, idesc, 1);
          }
        }
        mma_commit(&done);
      }
      __syncwarp();
      mbar_wait(&done, runs++ & 1, &abort_flag, p.status);
      tc_fence_after();
      __syncthreads();                     // (the warps reconverge before the TMEM loads)
      if (warp < 8 && nc + (warp & 3) * 32 < p.dv) {
        // a warp: 32 columns of 16 sequences
        const int half = warp >> 2, col = nc + (warp & 3) * 32 + lane;
        if (16 * half < n) {
          uint32_t v[16];
          tmem_ld16(tbase + ((uint32_t)((warp & 3) * 32) << 16) + 16 * half, v);
          tmem_wait_ld();
          if (col < p.dv) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int row = 16 * half + k;
              if (row >= n) break;
              const int64_t at = ((int64_t)(base + row) * p.h + hh) * p.dv + col;
              const float x = __uint_as_float(v[k]);
              const __nv_bfloat16 hi = __float2bfloat16(x);
              p.out[at] = hi;
              if (p.out_lo) p.out_lo[at] = __float2bfloat16(x - __bfloat162float(hi));
            }
          }
        }
      }
      tc_fence_before();
      __syncthreads();                     // TMEM and, past 128 columns, weights are read
      tc_fence_after();
    }
  }
  if (warp == 1) tmem_dealloc(tbase, 32);
}

// W_UK and W_UV rows of all heads, boxes of 128 rows x 64 columns.
bool weight_map(CUtensorMap* m, const PagedDecodeArgs& a) {
  const uint64_t dims[2] = {(uint64_t)R, (uint64_t)a.h * (a.dn + a.dv)}, str[1] = {R * 2};
  const uint32_t box[2] = {64, 128};
  return encode_tmap(m, a.w_kv_b, 2, dims, str, box);
}

}  // namespace

cudaError_t launch_paged_query(const PagedDecodeArgs& a, int min_len, cudaStream_t st) {
  CUtensorMap tmW;
  if (!weight_map(&tmW, a)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_query_kernel, Q_SMEM, set);
  if (e != cudaSuccess) return e;
  QueryParams q;
  q.q_nope = (const __nv_bfloat16*)a.q_nope;
  q.q_pe = (const __nv_bfloat16*)a.q_pe;
  q.q8 = a.q8; q.qf = a.qf; q.ctx = a.ctx; q.pre = a.pre; q.len = a.len;
  q.B = a.B; q.h = a.h; q.dn = a.dn; q.dv = a.dv;
  q.groups = a.tc.groups; q.hg_heads = a.tc.hg_heads; q.NH = a.tc.NH;
  q.first = a.first; q.parts = (int2*)a.parts; q.n_units = a.tc.n_units; q.min_len = min_len;
  q.most = (int64_t)a.max_blocks * a.pool.bs;
  q.scale_log2 = a.scale * 1.4426950408889634f;
  q.status = a.status;
  q.rounds = rounds_of(a);
  const int pads = q.groups * q.NH - q.h;
  count_launches();
  const dim3 grid(1 + a.h + pads, (a.B + MB * q.rounds - 1) / (MB * q.rounds));
  return launch_pdl(paged_query_kernel, grid, dim3(NT), Q_SMEM, st, tmW, q);
}

cudaError_t launch_paged_output(const PagedDecodeArgs& a, cudaStream_t st) {
  CUtensorMap tmW;
  if (!weight_map(&tmW, a)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_output_kernel, O_SMEM, set);
  if (e != cudaSuccess) return e;
  OutputParams o;
  o.part_o = a.part_o; o.part_lse = a.part_lse; o.o_lat = (const float*)a.o_lat;
  o.parts = (const int2*)a.parts;
  o.out = (__nv_bfloat16*)a.o; o.out_lo = (__nv_bfloat16*)a.o_lo;
  o.B = a.B; o.h = a.h; o.dn = a.dn; o.dv = a.dv;
  o.status = a.status;
  o.rounds = rounds_of(a);
  count_launches();
  return launch_pdl(paged_output_kernel, dim3(a.h, (a.B + MB * o.rounds - 1) / (MB * o.rounds)), dim3(NT),
                    O_SMEM, st, tmW, o);
}

}  // namespace mla
