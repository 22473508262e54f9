// CUDA-core weight-absorbed decode over the paged 8-bit latent cache, in fp32
// arithmetic.  With the values v_j = e4m3(byte) 2^e of a block's rows:
//   q_lat[b,h] = W_UK[h]^T q_nope[b,h]                       (absorb kernel)
//   s_j = scale (q_lat . c_j + q_pe . kpe_j); partial softmax
//   statistics and sums over splits of the context           (split kernel)
//   log-sum-exp merge of the splits, o = W_UV[h] o_lat       (merge kernel)
// Between the kernels q_lat, and o before an output projection, are in the
// model's type: with bf16 that is 2^-8 of each value, the precision that the
// query and the output have anyway, and the projections behind read bf16.
// Every head reads the rows again (from L2, mostly) and the products are fp32
// FMAs, so this is the form for what the tensor cores do not take: fp32 and
// other widths.  8 requests of up to 2000 tokens, 4 heads of a small fp32 layer:
// 13 us, which is three launches and their trips to memory.
#include "paged.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace paged;

template <typename T>
__global__ void paged_absorb_kernel(PagedDecodeArgs a) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    a.status[0] = a.status[1] = 0;
  const int b = blockIdx.x, hh = blockIdx.y;
  extern __shared__ float qn[];
  const T* qnope = reinterpret_cast<const T*>(a.q_nope) + ((int64_t)b * a.h + hh) * a.dn;
  for (int d = threadIdx.x; d < a.dn; d += blockDim.x) qn[d] = Elem<T>::load(qnope + d);
  __syncthreads();
  const T* W = reinterpret_cast<const T*>(a.w_kv_b) + (int64_t)hh * (a.dn + a.dv) * a.r;
  T* out = reinterpret_cast<T*>(a.q_lat) + ((int64_t)b * a.h + hh) * (a.r + a.dr);
  for (int c = threadIdx.x; c < a.r; c += blockDim.x) {
    float s = 0.f;
#pragma unroll 8
    for (int d = 0; d < a.dn; ++d) s = fmaf(qn[d], Elem<T>::load(W + (int64_t)d * a.r + c), s);
    Elem<T>::store(out + c, s);
  }
  const T* qpe = reinterpret_cast<const T*>(a.q_pe) + ((int64_t)b * a.h + hh) * a.dr;
  for (int c = threadIdx.x; c < a.dr; c += blockDim.x) out[a.r + c] = qpe[c];
}

// Cached tokens of sequence b, clamped to the table; out of range is reported.
__device__ __forceinline__ int tokens_of(const PagedDecodeArgs& a, int b) {
  const int n = a.ctx[b];
  const int64_t most = (int64_t)a.max_blocks * a.pool.bs;
  if (n >= 0 && n <= most) return n;
  if (threadIdx.x == 0) atomicOr(a.status, kStatusBadPage);
  return n < 0 ? 0 : (int)most;
}

// One block per (sequence, head, split of the context): four threads share a
// token's dot product (16-byte pieces in turn), then a thread owns four latent
// columns of every tl-th token.
constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_split_kernel(PagedDecodeArgs a) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int b = blockIdx.x, hh = blockIdx.y, sp = blockIdx.z, tid = threadIdx.x;
  const int n = tokens_of(a, b), t0 = sp * a.split_tokens;
  const int64_t part = ((int64_t)b * a.max_splits + sp) * a.h + hh;
  if (t0 >= n) {                              // empty split: the merge skips it
    if (tid == 0) a.part_lse[part] = -INFINITY;
    return;
  }
  const int nt = min(n - t0, a.split_tokens), w = a.pool.W, bs = a.pool.bs;
  extern __shared__ __align__(16) float sm[];
  float* q = sm;                              // [w]
  float* red = q + w;                         // [4 kThreads] sums of the token lanes
  float* s = red + 4 * kThreads;              // [split_tokens] scores, then weights
  float* scl = s + a.split_tokens;            // [split_tokens / 16] scale of every 16 tokens
  int* blk = reinterpret_cast<int*>(scl + a.split_tokens / 16);   // their block
  __shared__ float part_max[32], part_sum[32];
  const T* ql = reinterpret_cast<const T*>(a.q_lat) + ((int64_t)b * a.h + hh) * w;
  for (int g = tid; g < (nt + 15) / 16; g += kThreads) {
    int id = a.table[(int64_t)b * a.max_blocks + (t0 + 16 * g) / bs];
    if (id < 0 || id >= a.pool.n_blocks) {
      atomicOr(a.status, kStatusBadPage);
      id = 0;
    }
    blk[g] = id;
    scl[g] = read_scale(a.pool.scales[id], a.status);
  }
  for (int c = tid; c < w; c += kThreads) q[c] = Elem<T>::load(ql + c);
  __syncthreads();
  auto row = [&](int t) {
    return a.pool.cache + ((int64_t)blk[t >> 4] * bs + (t0 + t) % bs) * w;
  };
  const int warp = tid / 32, lane = tid % 32;
  float mx = -INFINITY;
  for (int tb = 0; tb < nt; tb += kThreads / 4) {
    const int t = tb + tid / 4;
    float acc = 0.f;
    if (t < nt) {
      const uint8_t* c8 = row(t);
      for (int c = (tid & 3) * 16; c < w; c += 64) {
        float v[16];
        dequant16(*reinterpret_cast<const uint4*>(c8 + c), 1.f, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(q + c + 4 * i);
          acc = fmaf(x.x, v[4 * i], acc);
          acc = fmaf(x.y, v[4 * i + 1], acc);
          acc = fmaf(x.z, v[4 * i + 2], acc);
          acc = fmaf(x.w, v[4 * i + 3], acc);
        }
      }
    }
    acc += __shfl_xor_sync(0xffffffffu, acc, 1);
    acc += __shfl_xor_sync(0xffffffffu, acc, 2);
    if (t < nt) {
      acc *= scl[t >> 4] * a.scale;
      if ((tid & 3) == 0) s[t] = acc;
      mx = fmaxf(mx, acc);
    }
  }
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) part_max[warp] = mx;
  __syncthreads();
  mx = -INFINITY;
  for (int i = 0; i < kThreads / 32; ++i) mx = fmaxf(mx, part_max[i]);
  float l = 0.f;
  for (int t = tid; t < nt; t += kThreads) {
    const float p = expf(s[t] - mx);
    s[t] = p * scl[t >> 4];                   // the weight of the row's e4m3 values
    l += p;
  }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) part_sum[warp] = l;
  __syncthreads();
  l = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) l += part_sum[i];
  if (tid == 0) a.part_lse[part] = mx + logf(l);
  const float inv = 1.f / l;
  // column groups of four in rounds of up to kThreads; r % 4 columns at the
  // end read past them into the rope part, which is not stored
  const int groups = (a.r + 3) / 4;
  for (int g0 = 0; g0 < groups; g0 += kThreads) {
    const int ng = min(groups - g0, kThreads), tl = kThreads / ng;
    const int cg = tid % ng, ti = tid / ng;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    if (ti < tl) {
      for (int t = ti; t < nt; t += tl) {
        float v[4];
        from_e4m3x4(*reinterpret_cast<const uint32_t*>(row(t) + 4 * (g0 + cg)), v);
        const float p = s[t];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = fmaf(p, v[k], o[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) red[(ti * ng + cg) * 4 + k] = o[k];
    }
    __syncthreads();
    for (int c = tid; c < 4 * ng; c += kThreads) {
      float x = 0.f;
      for (int i = 0; i < tl; ++i) x += red[i * ng * 4 + c];
      if (4 * g0 + c < a.r) a.part_o[part * a.r + 4 * g0 + c] = x * inv;
    }
    __syncthreads();
  }
}

// o_lat[b,h] from the splits (zero for a sequence without tokens), then
// o[b,h] = W_UV[h] o_lat; one block per (sequence, head).
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_merge_kernel(PagedDecodeArgs a) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int b = blockIdx.x, hh = blockIdx.y, tid = threadIdx.x;
  extern __shared__ __align__(16) float ol[];   // [r], then [kThreads] sums
  float* red = ol + a.r;
  __shared__ float part_max[32], part_den[32];
  const int warp = tid / 32, lane = tid % 32;
  const int n = tokens_of(a, b), ns = (n + a.split_tokens - 1) / a.split_tokens;
  const int64_t p0 = (int64_t)b * a.max_splits * a.h + hh;
  float mx = -INFINITY;
  for (int sp = tid; sp < ns; sp += kThreads)
    mx = fmaxf(mx, a.part_lse[p0 + (int64_t)sp * a.h]);
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) part_max[warp] = mx;
  __syncthreads();
  mx = -INFINITY;
  for (int i = 0; i < kThreads / 32; ++i) mx = fmaxf(mx, part_max[i]);
  float den = 0.f;                            // stays 0 without tokens; NaN passes through
  for (int sp = tid; sp < ns; sp += kThreads) den += expf(a.part_lse[p0 + (int64_t)sp * a.h] - mx);
  for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (lane == 0) part_den[warp] = den;
  __syncthreads();
  den = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) den += part_den[i];
  // rounds of up to kThreads columns; the threads left over share the splits
  for (int c0 = 0; c0 < a.r; c0 += kThreads) {
    const int nc = min(a.r - c0, kThreads), sl = kThreads / nc, c = tid % nc, si = tid / nc;
    float o = 0.f;
    if (si < sl)
      for (int sp = si; sp < ns; sp += sl) {
        const int64_t part = p0 + (int64_t)sp * a.h;
        o = fmaf(expf(a.part_lse[part] - mx), a.part_o[part * a.r + c0 + c], o);
      }
    red[tid] = o;
    __syncthreads();
    if (tid < nc) {
      float x = 0.f;
      for (int i = 0; i < sl; ++i) x += red[i * nc + tid];
      ol[c0 + tid] = ns == 0 ? 0.f : x / den;
    }
    __syncthreads();
  }
  const T* W = reinterpret_cast<const T*>(a.w_kv_b) + ((int64_t)hh * (a.dn + a.dv) + a.dn) * a.r;
  T* out = reinterpret_cast<T*>(a.o) + ((int64_t)b * a.h + hh) * a.dv;
  // four columns of a warp at a time, so that their loads are in flight together
  constexpr int G = 4;
  for (int v0 = G * warp; v0 < a.dv; v0 += G * kThreads / 32) {
    float acc[G];
    const int n = min(G, a.dv - v0);
#pragma unroll
    for (int k = 0; k < G; ++k) acc[k] = 0.f;
#pragma unroll 2
    for (int c = lane; c < a.r; c += 32) {
#pragma unroll
      for (int k = 0; k < G; ++k)
        if (k < n) acc[k] = fmaf(Elem<T>::load(W + (int64_t)(v0 + k) * a.r + c), ol[c], acc[k]);
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      for (int s = 16; s; s >>= 1) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], s);
      if (lane == 0 && k < n) Elem<T>::store(out + v0 + k, acc[k]);
    }
  }
}

// out = o W_o^T for a few rows, fp32: a warp per column of the output and up to
// ROWS sequences, the lanes sharing K.
constexpr int ROWS = 8;

__global__ void __launch_bounds__(kThreads)
    paged_oproj_simt_kernel(const float* __restrict__ o, const float* __restrict__ w_o,
                            float* __restrict__ out, int B, int K, int hidden) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int col = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
  const int b0 = blockIdx.y * ROWS, n = min(ROWS, B - b0);
  if (col >= hidden) return;
  const float* w = w_o + (int64_t)col * K;
  const float* x = o + (int64_t)b0 * K;
  float acc[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) acc[r] = 0.f;
#pragma unroll 2
  for (int k = lane; k < K; k += 32) {
    const float v = w[k];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (r < n) acc[r] = fmaf(v, x[(int64_t)r * K + k], acc[r]);
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    for (int s = 16; s; s >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], s);
    if (lane == 0 && r < n) out[(int64_t)(b0 + r) * hidden + col] = acc[r];
  }
}

template <typename T>
cudaError_t run(const PagedDecodeArgs& a, cudaStream_t st) {
  const dim3 bh(a.B, a.h);
  cudaError_t e =
      launch_pdl(paged_absorb_kernel<T>, bh, dim3(kThreads), a.dn * sizeof(float), st, a);
  count_launches();
  if (e != cudaSuccess) return e;
  stage_event(1, st);
  static std::atomic<uint64_t> set{0}, set_m{0};
  e = set_dynamic_smem((const void*)paged_split_kernel<T>, kMaxSmem, set);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_split_kernel<T>, dim3(a.B, a.h, a.max_splits), dim3(kThreads),
                 paged_simt_smem(a.r + a.dr, a.split_tokens), st, a);
  count_launches();
  if (e != cudaSuccess) return e;
  stage_event(2, st);
  e = set_dynamic_smem((const void*)paged_merge_kernel<T>, kMaxSmem, set_m);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_merge_kernel<T>, bh, dim3(kThreads), (a.r + kThreads) * sizeof(float), st, a);
  count_launches();
  if (e != cudaSuccess) return e;
  stage_event(3, st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_oproj_simt(const float* o, const float* w_o, float* out, int B, int K,
                                    int hidden, cudaStream_t st) {
  const dim3 grid((hidden + kThreads / 32 - 1) / (kThreads / 32), (B + ROWS - 1) / ROWS);
  count_launches();
  return launch_pdl(paged_oproj_simt_kernel, grid, dim3(kThreads), 0, st, o, w_o, out, B, K, hidden);
}

cudaError_t launch_paged_decode_simt(int dtype, const PagedDecodeArgs& a, cudaStream_t st) {
  return dtype == MLA_F32 ? run<float>(a, st) : run<__nv_bfloat16>(a, st);
}

}  // namespace mla
