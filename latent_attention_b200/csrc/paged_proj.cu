// The two projections around the tensor-core paged attention, one head and 32
// sequences a block:
//
//   paged_query_kernel   q_lat = W_UK[h]^T q_nope, and [q_lat | q_pe] as two
//                        e4m3 terms and a power of two; the lengths and the
//                        chunk line of all sequences
//   paged_output_kernel  o_lat of every sequence from its partial results, and
//                        o = W_UV[h] o_lat
//
// Both read each head's 128 KB of weights once and do little with them (a
// decode batch has tens of rows): what bounds them is the time of a launch and
// of one trip to memory, so the work around the products (rounding to 8 bits,
// merging) is done where the operands are, and the products are warp-level
// MMAs on shared memory, whose results the threads hold in registers; a
// tcgen05 product would have to be read back out of TMEM first.  Neither
// q_lat nor o_lat is rounded to 16 bits: q_lat goes from fp32 to its two
// terms, o_lat enters the product as two bf16 terms (16 significant bits).
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
constexpr int NT = 256;                  // threads, 8 warps
constexpr int MB = 32;                   // sequences a block
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
  int32_t* len;
  int B, h, dn, dv, groups, hg_heads, NH;
  int64_t most;                            // tokens a table holds
  float scale_log2;
  uint32_t* status;
};
constexpr int Q_STAGE = MB * 2 * W;        // the rows' bytes, both terms
constexpr int Q_SMEM = W_BYTES + Q_STAGE + 1024;

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
  if (t == 0) *p.status = 0;
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
}

// Block (x, y): x = 0 the lengths, 1 .. h a head, h + 1 the rows that pad the
// head groups; y: sequences 32 y ...
__global__ void __launch_bounds__(NT) paged_query_kernel(const __grid_constant__ CUtensorMap tmW,
                                                         QueryParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full;
  __shared__ int abort_flag;
  __shared__ uint32_t amax_s[MB][9];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    mbar_init(&full, 1);
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tmW);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int b0 = blockIdx.y * MB, nb = min(MB, p.B - b0);
  if (blockIdx.x == 0) {
    if (blockIdx.y == 0) lengths(p);
    return;
  }
  if ((int)blockIdx.x > p.h) {
    const int pad = p.groups * p.NH - p.h;
    for (int k = t; k < nb * pad * 2 * (W / 16); k += NT) {
      const int c = k % (W / 16), term = k / (W / 16) % 2, j = k / (W / 8) % pad;
      const int64_t b = b0 + k / (W / 8) / pad;
      // pad row j: groups are full but for the last rows of each
      int g = 0, i = j;
      for (; g < p.groups; ++g) {
        const int real = min(p.hg_heads, p.h - g * p.hg_heads), n = p.NH - real;
        if (i < n) { i += real; break; }
        i -= n;
      }
      const int64_t bg = b * p.groups + g;
      *reinterpret_cast<uint4*>(p.q8 + ((bg * 2 + term) * p.NH + i) * W + c * 16) =
          make_uint4(0u, 0u, 0u, 0u);
      if (c == 0 && term == 0) p.qf[bg * p.NH + i] = 0.f;
    }
    return;
  }
  const int hh = blockIdx.x - 1;
  const uint32_t wbase = smem_u32(smem);
  float acc[2][8][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[m][n][k] = 0.f;
  const int r = lane >> 2, kq = 2 * (lane & 3);
  bool ok = true;
  for (int kc = 0; kc < p.dn; kc += 128) {
    // 128 rows of W_UK[h]; past dn they are W_UV's and meet zeros of q
    if (t == 0) {
      mbar_arrive_expect_tx(&full, W_BYTES);
      for (int i = 0; i < 8; ++i)
        tma_load_2d(smem + i * WBOX, &tmW, 64 * i, hh * (p.dn + p.dv) + kc, &full);
    }
    uint32_t a[2][8][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = m * 16 + r + (q & 1) * 8, k = kc + ks * 16 + kq + (q >> 1) * 8;
          a[m][ks][q] =
              row < nb && k < p.dn
                  ? *reinterpret_cast<const uint32_t*>(
                        p.q_nope + ((int64_t)(b0 + row) * p.h + hh) * p.dn + k)
                  : 0u;
        }
    if (!mbar_wait(&full, (kc >> 7) & 1, &abort_flag, p.status)) { ok = false; break; }
    // this warp's 64 latent columns are one box
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t b[4];
        ldsm4_t(wbase + warp * WBOX + box_at(ks * 16 + (lane & 15), 2 * n + (lane >> 4)), b);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m * 16 >= nb) continue;
          mma16816(acc[m][2 * n], a[m][ks], b[0], b[1]);
          mma16816(acc[m][2 * n + 1], a[m][ks], b[2], b[3]);
        }
      }
    }
    __syncthreads();                       // the weights are read
  }
  if (!ok) return;                         // the status word says so
  // the rows' maxima
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x = 0;
#pragma unroll
      for (int n = 0; n < 8; ++n)
        x = max(x, max(finite_bits(acc[m][n][2 * half]), finite_bits(acc[m][n][2 * half + 1])));
      x = max(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = max(x, __shfl_xor_sync(0xffffffffu, x, 2));
      if ((lane & 3) == 0) amax_s[m * 16 + half * 8 + r][warp] = x;
    }
  const int rr = t >> 3, part = t & 7;     // eight threads a row for its rope part
  float pe[8];
  {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (rr < nb)
      x = reinterpret_cast<const uint4*>(p.q_pe + ((int64_t)(b0 + rr) * p.h + hh) * DR)[part];
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pe[2 * i] = __uint_as_float(xw[i] << 16);
      pe[2 * i + 1] = __uint_as_float(xw[i] & 0xffff0000u);
      m = max(m, max(finite_bits(pe[2 * i]), finite_bits(pe[2 * i + 1])));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (part == 0) amax_s[rr][8] = m;
  }
  __syncthreads();
  auto exponent = [&](int row) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) m = max(m, amax_s[row][i]);
    return scale_exp(m);
  };
  uint8_t* stage = smem + W_BYTES;         // [MB][2][W]
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = m * 16 + half * 8 + r;
      const float f = pow2(-exponent(row));
      uint8_t* dst = stage + row * 2 * W + warp * 64 + kq;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const uint32_t v = split_pair(acc[m][n][2 * half] * f, acc[m][n][2 * half + 1] * f);
        *reinterpret_cast<uint16_t*>(dst + 8 * n) = (uint16_t)v;
        *reinterpret_cast<uint16_t*>(dst + W + 8 * n) = (uint16_t)(v >> 16);
      }
    }
  const int g = hh / p.hg_heads, i = hh % p.hg_heads;
  {
    const int e = exponent(rr);
    const float f = pow2(-e);
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = split_pair(pe[2 * k] * f, pe[2 * k + 1] * f);
    uint8_t* dst = stage + rr * 2 * W + R + part * 8;
    *reinterpret_cast<uint2*>(dst) = make_uint2((v[0] & 0xffffu) | (v[1] << 16),
                                                (v[2] & 0xffffu) | (v[3] << 16));
    *reinterpret_cast<uint2*>(dst + W) = make_uint2((v[0] >> 16) | (v[1] & 0xffff0000u),
                                                    (v[2] >> 16) | (v[3] & 0xffff0000u));
    if (part == 0 && rr < nb)
      p.qf[((int64_t)(b0 + rr) * p.groups + g) * p.NH + i] = p.scale_log2 * pow2(e);
  }
  __syncthreads();
  for (int k = t; k < nb * 2 * (W / 16); k += NT) {
    const int row = k / (2 * (W / 16)), rest = k % (2 * (W / 16));
    const int term = rest / (W / 16), c = rest % (W / 16);
    const int64_t bg = (int64_t)(b0 + row) * p.groups + g;
    *reinterpret_cast<uint4*>(p.q8 + ((bg * 2 + term) * p.NH + i) * W + c * 16) =
        *reinterpret_cast<const uint4*>(stage + (row * 2 + term) * W + c * 16);
  }
}

// ------------------------------------------------------------------ output
struct OutputParams {
  const float *part_o, *part_lse;          // [2 n_units, h, R], [2 n_units, h] (log2)
  const float* o_lat;                      // [B, h, R]: sequences in one segment
  const int64_t* pre;
  __nv_bfloat16* out;                      // [B, h, dv]
  int B, h, dn, dv, n_units, min_len;
  uint32_t* status;
};
constexpr int A_BYTES = 8 * MB * 128;      // o_lat of the block's sequences, one bf16 term
constexpr int O_RED = 8 * R * 4;
constexpr int O_SMEM = W_BYTES + 2 * A_BYTES + O_RED + 1024;
constexpr int kUnits = 512;               // most units (host side: tc_paged_plan)
constexpr int kShared = 4;                 // more partials than this: the whole block merges

__global__ void __launch_bounds__(NT) paged_output_kernel(const __grid_constant__ CUtensorMap tmW,
                                                          OutputParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full;
  __shared__ int abort_flag;
  __shared__ uint32_t many;                // rows that the whole block merges
  __shared__ float w_s[2 * kUnits];        // lse and weights of one such row's partials
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int hh = blockIdx.x, b0 = blockIdx.y * MB, nb = min(MB, p.B - b0);
  const uint32_t wbase = smem_u32(smem), abase = wbase + W_BYTES;
  float* red = reinterpret_cast<float*>(smem + W_BYTES + 2 * A_BYTES);
  if (t == 0) {
    mbar_init(&full, 1);
    abort_flag = 0;
    many = 0;
    fence_barrier_init();
    // The weights do not depend on the kernel before this one (which started
    // only once all before it had finished): they are on their way while it
    // ends.
    mbar_arrive_expect_tx(&full, W_BYTES);
    for (int i = 0; i < 8; ++i)
      tma_load_2d(smem + i * WBOX, &tmW, 64 * i, hh * (p.dn + p.dv) + p.dn, &full);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // 16 dims of a row as two bf16 terms into the A operand's boxes
  auto put = [&](int row, int at16, const float (&v)[16]) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      lo[i] = pack_bf16(v[2 * i] - __uint_as_float(hi[i] << 16),
                        v[2 * i + 1] - __uint_as_float(hi[i] & 0xffff0000u));
    }
    const uint32_t box = abase + (at16 >> 2) * MB * 128;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t at = box + box_at(row, 2 * (at16 & 3) + q);
      st_shared_v4(at, hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
      st_shared_v4(at + A_BYTES, lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
    }
  };
  for (int row = warp; row < MB; row += NT / 32) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    const int b = b0 + row;
    if (row < nb && p.pre[b + 1] != p.pre[b]) {
      const SeqUnits su = seq_units(p.pre, b, p.B, p.n_units, p.min_len);
      if (su.u0 == su.u1) {
        load16(p.o_lat + ((int64_t)b * p.h + hh) * R + lane * 16, v);
      } else if (su.u1 - su.u0 < kShared) {
        float mx = -INFINITY, den = 0.f, lse[kShared];
#pragma unroll
        for (int i = 0; i < kShared; ++i) {
          lse[i] = su.u0 + i <= su.u1
                       ? p.part_lse[(int64_t)seq_slot(su, su.u0 + i) * p.h + hh] : -INFINITY;
          mx = fmaxf(mx, lse[i]);
        }
#pragma unroll
        for (int i = 0; i < kShared; ++i) {
          if (su.u0 + i > su.u1) break;
          const float w = exp2f(lse[i] - mx);
          float x[16];
          load16(p.part_o + ((int64_t)seq_slot(su, su.u0 + i) * p.h + hh) * R + lane * 16, x);
          den += w;
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = fmaf(w, x[k], v[k]);
        }
        const float inv = 1.f / den;
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] *= inv;
      } else {
        if (lane == 0) atomicOr(&many, 1u << row);
        continue;
      }
    }
    put(row, lane, v);
  }
  __syncthreads();
  for (uint32_t left = many; left; left &= left - 1) {
    const int row = __ffs(left) - 1, b = b0 + row;
    const SeqUnits su = seq_units(p.pre, b, p.B, p.n_units, p.min_len);
    const int n = su.u1 - su.u0 + 1;       // at most kUnits
    float mx = -INFINITY;
    for (int i = lane; i < n; i += 32) {
      const float x = p.part_lse[(int64_t)seq_slot(su, su.u0 + i) * p.h + hh];
      if (warp == 0) w_s[i] = x;
      mx = fmaxf(mx, x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    __syncthreads();
    for (int i = t; i < n; i += NT) w_s[kUnits + i] = exp2f(w_s[i] - mx);
    __syncthreads();
    float v[16], den = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = 0.f;
#pragma unroll 2
    for (int i = warp; i < n; i += NT / 32) {
      float x[16];
      load16(p.part_o + ((int64_t)seq_slot(su, su.u0 + i) * p.h + hh) * R + lane * 16, x);
      const float w = w_s[kUnits + i];
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = fmaf(w, x[k], v[k]);
    }
    store16(red + warp * R + lane * 16, v);
    for (int i = lane; i < n; i += 32) den += w_s[kUnits + i];
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    __syncthreads();
    if (warp == 0) {
      const float inv = 1.f / den;
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = 0.f;
      for (int w = 0; w < NT / 32; ++w) {
        float x[16];
        load16(red + w * R + lane * 16, x);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] += x[k];
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= inv;
      put(row, lane, v);
    }
    __syncthreads();
  }
  for (int nc = 0; nc < p.dv; nc += 128) {
    if (nc > 0 && t == 0) {
      mbar_arrive_expect_tx(&full, W_BYTES);
      for (int i = 0; i < 8; ++i)
        tma_load_2d(smem + i * WBOX, &tmW, 64 * i, hh * (p.dn + p.dv) + p.dn + nc, &full);
    }
    if (!mbar_wait(&full, (nc >> 7) & 1, &abort_flag, p.status)) return;
    const int n0 = warp * 16;              // this warp's rows of W_UV
    if (nc + n0 < p.dv) {
      float acc[2][2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][n][k] = 0.f;
#pragma unroll 4
      for (int ks = 0; ks < R / 16; ++ks) {
        const int box = ks >> 2, c = 2 * (ks & 3);
        uint32_t b[4];
        ldsm4(wbase + box * WBOX +
                  box_at(n0 + (lane & 7) + ((lane >> 4) & 1) * 8, c + ((lane >> 3) & 1)), b);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m * 16 >= nb) continue;
          const uint32_t at = abase + box * MB * 128 + box_at(m * 16 + (lane & 15), c + (lane >> 4));
          uint32_t hi[4], lo[4];
          ldsm4(at, hi);
          ldsm4(at + A_BYTES, lo);
          mma16816(acc[m][0], lo, b[0], b[1]);
          mma16816(acc[m][1], lo, b[2], b[3]);
          mma16816(acc[m][0], hi, b[0], b[1]);
          mma16816(acc[m][1], hi, b[2], b[3]);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = m * 16 + half * 8 + (lane >> 2);
            const int col = nc + n0 + n * 8 + 2 * (lane & 3);
            if (row < nb && col < p.dv)
              *reinterpret_cast<uint32_t*>(p.out + ((int64_t)(b0 + row) * p.h + hh) * p.dv + col) =
                  pack_bf16(acc[m][n][2 * half], acc[m][n][2 * half + 1]);
          }
    }
    __syncthreads();                       // the weights are read
  }
}

// W_UK and W_UV rows of all heads, boxes of 128 rows x 64 columns.
bool weight_map(CUtensorMap* m, const PagedDecodeArgs& a) {
  const uint64_t dims[2] = {(uint64_t)R, (uint64_t)a.h * (a.dn + a.dv)}, str[1] = {R * 2};
  const uint32_t box[2] = {64, 128};
  return encode_tmap(m, a.w_kv_b, 2, dims, str, box);
}

}  // namespace

cudaError_t launch_paged_query(const PagedDecodeArgs& a, cudaStream_t st) {
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
  q.most = (int64_t)a.max_blocks * a.pool.bs;
  q.scale_log2 = a.scale * 1.4426950408889634f;
  q.status = a.status;
  const bool pads = q.groups * q.NH > q.h;
  count_launches();
  return launch_pdl(paged_query_kernel, dim3(1 + a.h + pads, (a.B + MB - 1) / MB), dim3(NT), Q_SMEM,
                    st, tmW, q);
}

cudaError_t launch_paged_output(const PagedDecodeArgs& a, int min_len, cudaStream_t st) {
  CUtensorMap tmW;
  if (!weight_map(&tmW, a)) return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_output_kernel, O_SMEM, set);
  if (e != cudaSuccess) return e;
  OutputParams o;
  o.part_o = a.part_o; o.part_lse = a.part_lse; o.o_lat = (const float*)a.o_lat; o.pre = a.pre;
  o.out = (__nv_bfloat16*)a.o;
  o.B = a.B; o.h = a.h; o.dn = a.dn; o.dv = a.dv; o.n_units = a.tc.n_units; o.min_len = min_len;
  o.status = a.status;
  count_launches();
  return launch_pdl(paged_output_kernel, dim3(a.h, (a.B + MB - 1) / MB), dim3(NT), O_SMEM, st, tmW,
                    o);
}

}  // namespace mla
