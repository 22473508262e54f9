// CUDA-core weight-absorbed decode over the paged 8-bit latent cache, in fp32
// arithmetic.  With the values v_j = e4m3(byte) 2^e of a block's rows:
//   q_lat[b,h] = W_UK[h]^T q_nope[b,h]                       (absorb kernel)
//   s_j = scale (q_lat . c_j + q_pe . kpe_j); partial softmax
//   statistics and sums over splits of the context           (split kernel)
//   log-sum-exp merge of the splits, o = W_UV[h] o_lat       (merge kernel)
#include "paged.cuh"

namespace mla {
namespace {

using namespace paged;

template <typename T>
__global__ void paged_absorb_kernel(PagedDecodeArgs a) {
  const int b = blockIdx.x, hh = blockIdx.y;
  extern __shared__ float qn[];
  const T* qnope = reinterpret_cast<const T*>(a.q_nope) + ((int64_t)b * a.h + hh) * a.dn;
  for (int d = threadIdx.x; d < a.dn; d += blockDim.x) qn[d] = Elem<T>::load(qnope + d);
  __syncthreads();
  const T* W = reinterpret_cast<const T*>(a.w_kv_b) + (int64_t)hh * (a.dn + a.dv) * a.r;
  T* out = reinterpret_cast<T*>(a.q_lat) + ((int64_t)b * a.h + hh) * (a.r + a.dr);
  for (int c = threadIdx.x; c < a.r; c += blockDim.x) {
    float s = 0.f;
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

// One block per (sequence, head, split): the split's rows are found once, a
// warp scores a token, then every thread owns latent columns.
template <typename T>
__global__ void paged_split_kernel(PagedDecodeArgs a) {
  const int b = blockIdx.x, hh = blockIdx.y, sp = blockIdx.z;
  const int n = tokens_of(a, b), t0 = sp * a.split_tokens;
  const int64_t part = ((int64_t)b * a.max_splits + sp) * a.h + hh;
  if (t0 >= n) {                              // empty split: neutral partial
    for (int c = threadIdx.x; c < a.r; c += blockDim.x) a.part_o[part * a.r + c] = 0.f;
    if (threadIdx.x == 0) a.part_lse[part] = -INFINITY;
    return;
  }
  const int nt = min(n - t0, a.split_tokens), w = a.pool.W, bs = a.pool.bs;
  extern __shared__ float sm[];
  float* q = sm;                              // [w]
  float* s = q + w;                           // [split_tokens] scores, then weights
  float* scl = s + a.split_tokens;            // [split_tokens / 16] scale of every 16 tokens
  int* blk = reinterpret_cast<int*>(scl + a.split_tokens / 16);   // their block
  __shared__ float red[32];
  const T* ql = reinterpret_cast<const T*>(a.q_lat) + ((int64_t)b * a.h + hh) * w;
  for (int c = threadIdx.x; c < w; c += blockDim.x) q[c] = Elem<T>::load(ql + c);
  for (int g = threadIdx.x; g < (nt + 15) / 16; g += blockDim.x) {
    int id = a.table[(int64_t)b * a.max_blocks + (t0 + 16 * g) / bs];
    if (id < 0 || id >= a.pool.n_blocks) {
      atomicOr(a.status, kStatusBadPage);
      id = 0;
    }
    blk[g] = id;
    scl[g] = a.pool.scales[id];
  }
  __syncthreads();
  auto row = [&](int t) {
    return a.pool.cache + ((int64_t)blk[t >> 4] * bs + (t0 + t) % bs) * w;
  };
  auto value = [](const uint8_t* p) {
    float f[4];
    from_e4m3x4(*p, f);
    return f[0];
  };
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
  for (int t = warp; t < nt; t += nw) {
    const uint8_t* c8 = row(t);
    float acc = 0.f;
    for (int c = lane; c < w; c += 32) acc = fmaf(q[c], value(c8 + c), acc);
    for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) s[t] = acc * scl[t >> 4] * a.scale;
  }
  __syncthreads();
  float mx = -INFINITY;
  for (int t = threadIdx.x; t < nt; t += blockDim.x) mx = fmaxf(mx, s[t]);
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) red[warp] = mx;
  __syncthreads();
  mx = -INFINITY;
  for (int i = 0; i < nw; ++i) mx = fmaxf(mx, red[i]);
  __syncthreads();
  float l = 0.f;
  for (int t = threadIdx.x; t < nt; t += blockDim.x) {
    const float p = expf(s[t] - mx);
    s[t] = p * scl[t >> 4];                   // the weight of the row's e4m3 values
    l += p;
  }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[warp] = l;
  __syncthreads();
  l = 0.f;
  for (int i = 0; i < nw; ++i) l += red[i];
  for (int c = threadIdx.x; c < a.r; c += blockDim.x) {
    float o = 0.f;
    for (int t = 0; t < nt; ++t) o = fmaf(s[t], value(row(t) + c), o);
    a.part_o[part * a.r + c] = o / l;
  }
  if (threadIdx.x == 0) a.part_lse[part] = mx + logf(l);
}

// o_lat[b,h] from the splits (zero for a sequence without tokens), then
// o[b,h] = W_UV[h] o_lat; one block per (sequence, head).
template <typename T>
__global__ void paged_merge_kernel(PagedDecodeArgs a) {
  const int b = blockIdx.x, hh = blockIdx.y;
  extern __shared__ float ol[];               // [r]
  const int64_t p0 = (int64_t)b * a.max_splits * a.h + hh;
  float mx = -INFINITY;
  for (int sp = 0; sp < a.max_splits; ++sp) mx = fmaxf(mx, a.part_lse[p0 + (int64_t)sp * a.h]);
  float den = 0.f;                            // stays 0 without tokens; NaN passes through
  for (int sp = 0; sp < a.max_splits; ++sp) {
    const float l = a.part_lse[p0 + (int64_t)sp * a.h];
    den += l == -INFINITY ? 0.f : expf(l - mx);
  }
  for (int c = threadIdx.x; c < a.r; c += blockDim.x) {
    float o = 0.f;
    for (int sp = 0; sp < a.max_splits; ++sp) {
      const int64_t part = p0 + (int64_t)sp * a.h;
      const float l = a.part_lse[part];
      if (l != -INFINITY) o = fmaf(expf(l - mx), a.part_o[part * a.r + c], o);
    }
    ol[c] = den == 0.f ? 0.f : o / den;
  }
  __syncthreads();
  const T* W = reinterpret_cast<const T*>(a.w_kv_b) + ((int64_t)hh * (a.dn + a.dv) + a.dn) * a.r;
  T* out = reinterpret_cast<T*>(a.o) + ((int64_t)b * a.h + hh) * a.dv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, nw = blockDim.x / 32;
  for (int v = warp; v < a.dv; v += nw) {
    float acc = 0.f;
    for (int c = lane; c < a.r; c += 32)
      acc = fmaf(Elem<T>::load(W + (int64_t)v * a.r + c), ol[c], acc);
    for (int s = 16; s; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if (lane == 0) Elem<T>::store(out + v, acc);
  }
}

template <typename T>
cudaError_t run(const PagedDecodeArgs& a, cudaStream_t st) {
  const dim3 bh(a.B, a.h);
  paged_absorb_kernel<T><<<bh, 256, a.dn * sizeof(float), st>>>(a);
  stage_event(1, st);
  const int smem = paged_simt_smem(a.r + a.dr, a.split_tokens);
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_split_kernel<T>, kMaxSmem, set);
  if (e != cudaSuccess) return e;
  paged_split_kernel<T><<<dim3(a.B, a.h, a.max_splits), 256, smem, st>>>(a);
  stage_event(2, st);
  static std::atomic<uint64_t> set_m{0};
  const cudaError_t em = set_dynamic_smem((const void*)paged_merge_kernel<T>, kMaxSmem, set_m);
  if (em != cudaSuccess) return em;
  paged_merge_kernel<T><<<bh, 256, a.r * sizeof(float), st>>>(a);
  stage_event(3, st);
  count_launches(3);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_decode_simt(int dtype, const PagedDecodeArgs& a, cudaStream_t st) {
  return dtype == MLA_F32 ? run<float>(a, st) : run<__nv_bfloat16>(a, st);
}

}  // namespace mla
