// The paged 8-bit latent cache: block tables and slot maps from request
// lengths (plan), the quantised write by slot map (append), and the way back
// to rows of the model's type (gather).
//
// Megatron-LM MLA guide, 推理优化: a cached token keeps [kv_compressed |
// k_pos_emb].  Here the rows of all requests live in one pool of blocks of bs
// rows; a block holds e4m3 values and one power-of-two scale, so the value of
// a byte is e4m3(byte) * 2^e.  A power of two costs e4m3 nothing (its
// precision is relative) and makes moving a block to a larger scale an exponent
// shift: only values that become subnormal are rounded again.
#include <climits>

#include "paged.cuh"

namespace mla {
namespace {

using namespace paged;

// ------------------------------------------------------------------- plan
//
// held = ceil(ctx / bs), want = ceil((ctx + new) / bs), add = want - held
// blocks from the front of the free ring, in request order; a request with
// new = -1 gives its held blocks back behind the ring's end.  Blocks given
// back can be taken from the next call on, so the two never meet.
//
// One block of 1024 threads: the three prefix sums over the requests are a
// scan in registers and shared memory, and the entries that change hands are
// spread flat over the threads (a binary search in the prefix finds an
// entry's request), so one long prompt costs no more than many short ones.
// All or nothing: if anything is out of range or the ring or the slot map is
// too short, every output says "nothing happened".

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int wrap(int64_t i, int n) { return (int)(i >= n ? i - n : i); }

__device__ __forceinline__ void write_slot(const PlanArgs& a, int i, int total, const int32_t* ends,
                                           const int32_t* after) {
  int slot = -1, at = 0;
  if (i < total) {
    const int b = request_of(ends, a.B, i);
    at = after[b] - (ends[b] - i);               // the request's last new token is after[b] - 1
    const int blk = a.table[(int64_t)b * a.max_blocks + at / a.bs];
    if (blk >= 0 && blk < a.n_blocks) slot = blk * a.bs + at % a.bs;
    else atomicOr(a.status, kStatusBadPage);
  }
  a.slots[i] = slot;
  if (a.pos) a.pos[i] = at;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a, int inline_slots) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_sum[3][32];
  __shared__ int64_t totals[3];
  __shared__ int32_t s_head, s_count;
  int32_t *add_end = sm, *give_end = sm + a.B, *new_end = sm + 2 * a.B, *held = sm + 3 * a.B,
          *after = sm + 4 * a.B;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    s_head = a.state[0];
    s_count = a.state[1];
    *a.status = 0;
  }
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = t * per, b1 = min(b0 + per, a.B);
  int64_t add = 0, give = 0, fresh = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = a.ctx[b], n = a.fresh[b];
    const int64_t grow = n > 0 ? n : 0;
    int64_t hb = (c + a.bs - 1) / a.bs, wb = (c + grow + a.bs - 1) / a.bs;
    if (c < 0 || n < -1 || wb > a.max_blocks) { bad = true; hb = wb = 0; }
    add += n < 0 ? 0 : wb - hb;
    give += n < 0 ? hb : 0;
    fresh += grow;
    held[b] = (int)hb;
    after[b] = n < 0 ? 0 : (int)(c + grow);
    // inclusive within this thread; the threads before it are added below
    add_end[b] = (int)add;
    give_end[b] = (int)give;
    new_end[b] = (int)fresh;
  }
  const int64_t ia = warp_scan(add, lane), ig = warp_scan(give, lane), in = warp_scan(fresh, lane);
  if (lane == 31) {
    warp_sum[0][warp] = ia;
    warp_sum[1][warp] = ig;
    warp_sum[2][warp] = in;
  }
  const int any_bad = __syncthreads_or(bad);
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int64_t v = warp_sum[k][lane], s = warp_scan(v, lane);
      warp_sum[k][lane] = s - v;
      if (lane == 31) totals[k] = s;
    }
  }
  __syncthreads();
  const int64_t ta = totals[0], tg = totals[1], tn = totals[2];
  const int head = s_head, count = s_count, n = a.n_blocks;
  const bool broken = any_bad || head < 0 || head >= n || count < 0 || count > n ||
                      count + tg > n;            // more blocks than the pool has
  const bool ok = !broken && ta <= count && tn <= a.capacity;
  // exclusive prefix of this thread's requests (int: used only when ok)
  const int xa = (int)(warp_sum[0][warp] + ia - add), xg = (int)(warp_sum[1][warp] + ig - give),
            xn = (int)(warp_sum[2][warp] + in - fresh);
  for (int b = b0; b < b1; ++b) {
    add_end[b] += xa;
    give_end[b] += xg;
    new_end[b] += xn;
    a.cu[b + 1] = ok ? new_end[b] : 0;
    const int32_t was = a.ctx[b];                // before ctx_out, which may be ctx
    a.ctx_out[b] = ok ? after[b] : was;
  }
  if (t == 0) {
    a.cu[0] = 0;
    a.state_out[0] = ok ? wrap((int64_t)head + ta, n) : head;
    a.state_out[1] = ok ? (int)(count - ta + tg) : count;
    if (!ok) atomicOr(a.status, broken ? kStatusBadPage : kStatusNoBlocks);
  }
  __syncthreads();
  if (ok) {
    for (int i = t; i < (int)ta; i += kPlanThreads) {
      const int b = request_of(add_end, a.B, i);
      const int first = b ? add_end[b - 1] : 0;
      const int v = a.ring[wrap((int64_t)head + i, n)];
      if (v < 0 || v >= n) atomicOr(a.status, kStatusBadPage);
      a.table[(int64_t)b * a.max_blocks + held[b] + i - first] = v;
    }
    for (int i = t; i < (int)tg; i += kPlanThreads) {
      const int b = request_of(give_end, a.B, i);
      const int first = b ? give_end[b - 1] : 0;
      const int v = a.table[(int64_t)b * a.max_blocks + i - first];
      if (v < 0 || v >= n) atomicOr(a.status, kStatusBadPage);
      a.ring[wrap(wrap((int64_t)head + count, n) + (int64_t)i, n)] = v;
    }
  }
  if (inline_slots) {
    __syncthreads();
    for (int i = t; i < a.capacity; i += kPlanThreads)
      write_slot(a, i, ok ? (int)tn : 0, new_end, after);
  }
}

// The slot map on its own grid, from the plan's cu and lengths.
__global__ void slots_kernel(PlanArgs a) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < a.capacity) write_slot(a, i, a.cu[a.B], a.cu + 1, a.ctx_out);
}

// ----------------------------------------------------------------- append
//
// A run is a maximal stretch of rows whose slots are consecutive in one
// block; one CTA quantises it:  e = min{e : max|row| <= 448 2^e}; rows of the
// block in front of the run (offsets below its first slot) are kept and moved
// to max(e, e_old).  Rows behind the run are dead and stay as they were.
// A CTA takes the runs that start in its window of the slot map.
constexpr int kAppendThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const T* __restrict__ rows, const int32_t* __restrict__ slots, int n_rows,
                  PagedPool pool, int window, uint32_t* status, uint32_t* claims) {
  __shared__ int s_count, s_blk, s_off;     // run length (0: no run), its block and first row
  __shared__ uint32_t s_amax, s_odd;        // largest finite |value|, any NaN or infinity
  const int t = threadIdx.x, W = pool.W, bs = pool.bs;
  const int64_t n_slots = (int64_t)pool.n_blocks * bs;
  const int w0 = blockIdx.x * window, w1 = min(w0 + window, n_rows);
  for (int i = w0; i < w1; ++i) {
    __syncthreads();                         // the previous run's shared values are read
    if (t < 32) {
      const int s = slots[i], before = i > 0 ? slots[i - 1] : -1;
      const bool in = s >= 0 && s < n_slots;
      // a row of the block that the row before it writes: part of that run,
      // or (not its next slot) refused
      const bool cont = in && before >= 0 && before / bs == s / bs;
      if (t == 0) {
        s_count = 0;
        s_amax = 0;
        s_odd = 0;
        if ((!in && s != -1) || (cont && before + 1 != s)) atomicOr(status, kStatusBadPage);
      }
      if (in && !cont) {
        const int blk = s / bs, off = s % bs, most = min(bs - off, n_rows - i);
        int cnt = most;
        for (int k = 0; k < most; k += 32) {
          const bool same = k + t < most && slots[i + k + t] == s + k + t;
          const uint32_t m = __ballot_sync(0xffffffffu, same);
          if (m != 0xffffffffu) { cnt = k + __ffs(~m) - 1; break; }
        }
        if (t == 0) {
          // two runs of one call in one block have no order: the second is refused
          const uint32_t bit = 1u << (blk & 31);
          if (atomicOr(&claims[blk >> 5], bit) & bit) {
            atomicOr(status, kStatusBadPage);
          } else {
            s_count = cnt;
            s_blk = blk;
            s_off = off;
          }
        }
      }
    }
    __syncthreads();
    const int cnt = s_count;
    if (cnt == 0) continue;
    const int blk = s_blk, off = s_off;
    const T* src = rows + (int64_t)i * W;
    const int nv = cnt * W / 16;
    uint32_t amax = 0, odd = 0;
    for (int k = t; k < nv; k += kAppendThreads) {
      float v[16];
      load16(src + (int64_t)k * 16, v);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const uint32_t b = __float_as_uint(v[x]) & 0x7fffffffu;
        if (b < 0x7f800000u) amax = max(amax, b); else odd = 1;
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    odd = __reduce_or_sync(0xffffffffu, odd);
    if ((t & 31) == 0) {
      atomicMax(&s_amax, amax);
      if (odd) atomicOr(&s_odd, 1u);
    }
    __syncthreads();
    int e = scale_exp(s_amax), e_old = e;
    uint8_t* base = pool.cache + (int64_t)blk * bs * W;
    if (off > 0) {
      if (stored_exp(pool.scales[blk], &e_old)) {
        e = max(e, e_old);
      } else {
        if (t == 0) atomicOr(status, kStatusBadPage);
        e_old = e;
      }
    }
    if (e != e_old) {                        // the kept rows move to the larger scale
      const float f = pow2(e_old - e);
      uint4* kept = reinterpret_cast<uint4*>(base);
      for (int k = t; k < off * W / 16; k += kAppendThreads) {
        float v[16];
        dequant16(kept[k], f, v);
        kept[k] = make_uint4(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]),
                             to_e4m3x4(v[8], v[9], v[10], v[11]),
                             to_e4m3x4(v[12], v[13], v[14], v[15]));
      }
    }
    const float f = pow2(-e);
    uint4* dst = reinterpret_cast<uint4*>(base + (int64_t)off * W);
    const bool any_odd = s_odd != 0;
    for (int k = t; k < nv; k += kAppendThreads) {
      float v[16];
      load16(src + (int64_t)k * 16, v);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        // an infinity is stored as NaN, not as 448: x - x is NaN for both
        if (any_odd) v[x] += v[x] - v[x];
        v[x] *= f;
      }
      dst[k] = make_uint4(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]),
                          to_e4m3x4(v[8], v[9], v[10], v[11]),
                          to_e4m3x4(v[12], v[13], v[14], v[15]));
    }
    __syncthreads();                         // every thread has read the old scale
    if (t == 0) pool.scales[blk] = pow2(e);
  }
}

// ----------------------------------------------------------------- gather
//
// Rows of all requests back to back, and their prefix sums.  Each CTA scans
// the lengths into shared memory and takes tiles of kGatherRows rows: the
// tile's source rows are looked up once, then the tile is a flat list of
// 16-byte pieces.
constexpr int kGatherThreads = 256, kGatherRows = 64;

template <typename T>
__global__ void __launch_bounds__(kGatherThreads)
    gather_kernel(PagedPool pool, const int32_t* __restrict__ table,
                  const int32_t* __restrict__ ctx, T* __restrict__ rows, int32_t* __restrict__ cu,
                  int B, int max_blocks, int capacity, uint32_t* status) {
  extern __shared__ int32_t ends[];          // [B] inclusive prefix sums
  __shared__ int64_t warp_sum[kGatherThreads / 32];
  __shared__ int64_t src[kGatherRows];       // byte offset of the tile's rows, or -1
  __shared__ float scl[kGatherRows];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t most = (int64_t)max_blocks * pool.bs;
  const int per = (B + kGatherThreads - 1) / kGatherThreads;
  const int b0 = min(t * per, B), b1 = min(b0 + per, B);
  int64_t sum = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    int64_t n = ctx[b];
    if (n < 0 || n > most) { bad = true; n = n < 0 ? 0 : most; }
    sum += n;
  }
  const int64_t inc = warp_scan(sum, lane);
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t at = inc - sum;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int b = b0; b < b1; ++b) {
    int64_t n = ctx[b];
    n = n < 0 ? 0 : n > most ? most : n;
    at += n;
    ends[b] = (int32_t)(at < INT32_MAX ? at : INT32_MAX);
    if (blockIdx.x == 0) cu[b + 1] = ends[b];
  }
  __syncthreads();
  const int total = ends[B - 1];
  if (blockIdx.x == 0) {
    if (bad || (t == 0 && total > capacity)) atomicOr(status, kStatusBadPage);
    if (t == 0) cu[0] = 0;
  }
  const int n_rows = min(total, capacity), nv = pool.W / 16;
  for (int r0 = blockIdx.x * kGatherRows; r0 < n_rows; r0 += gridDim.x * kGatherRows) {
    if (t < kGatherRows) {
      int64_t o = -1;
      if (r0 + t < n_rows) {
        const int b = request_of(ends, B, r0 + t);
        const int j = r0 + t - (b ? ends[b - 1] : 0);
        const int blk = table[(int64_t)b * max_blocks + j / pool.bs];
        if (blk >= 0 && blk < pool.n_blocks) {
          o = ((int64_t)blk * pool.bs + j % pool.bs) * pool.W;
          scl[t] = pool.scales[blk];
        } else {
          atomicOr(status, kStatusBadPage);
        }
      }
      src[t] = o;
    }
    __syncthreads();
    const int pieces = min(kGatherRows, n_rows - r0) * nv;
    for (int k = t; k < pieces; k += kGatherThreads) {
      const int r = k / nv, c = (k - r * nv) * 16;
      float v[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) v[x] = 0.f;  // a row whose block is out of range
      if (src[r] >= 0)
        dequant16(*reinterpret_cast<const uint4*>(pool.cache + src[r] + c), scl[r], v);
      store16(rows + (int64_t)(r0 + r) * pool.W + c, v);
    }
    __syncthreads();
  }
}

// Slots that the planning block writes itself; beyond, a second grid does.
constexpr int kInlineSlots = 4096;

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  const int smem = 5 * 4 * a.B;
  static std::atomic<uint64_t> set{0};
  cudaError_t e = set_dynamic_smem((const void*)plan_kernel, 5 * 4 * kMaxRequests, set);
  if (e != cudaSuccess) return e;
  const bool in = a.capacity <= kInlineSlots;
  plan_kernel<<<1, kPlanThreads, smem, st>>>(a, in);
  count_launches();
  if (!in) {
    slots_kernel<<<(a.capacity + 255) / 256, 256, 0, st>>>(a);
    count_launches();
  }
  return cudaGetLastError();
}

cudaError_t launch_paged_append(int dtype, const void* rows, const int32_t* slots, int n_rows,
                                const PagedPool& pool, uint32_t* status, uint32_t* claims,
                                cudaStream_t st) {
  int window = (n_rows + 4 * 148 - 1) / (4 * 148);
  if (window > pool.bs) window = pool.bs;
  const int grid = (n_rows + window - 1) / window;
  count_launches();
  if (dtype == MLA_F32)
    append_kernel<float><<<grid, kAppendThreads, 0, st>>>((const float*)rows, slots, n_rows, pool,
                                                          window, status, claims);
  else
    append_kernel<__nv_bfloat16><<<grid, kAppendThreads, 0, st>>>(
        (const __nv_bfloat16*)rows, slots, n_rows, pool, window, status, claims);
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(int dtype, const PagedPool& pool, const int32_t* table,
                                const int32_t* ctx, void* rows, int32_t* cu, int B,
                                int max_blocks, int capacity, uint32_t* status, cudaStream_t st) {
  const int tiles = (capacity + kGatherRows - 1) / kGatherRows;
  const int grid = tiles < 8 * 148 ? (tiles > 0 ? tiles : 1) : 8 * 148;
  const size_t smem = 4 * (size_t)B;
  count_launches();
  if (dtype == MLA_F32)
    gather_kernel<float><<<grid, kGatherThreads, smem, st>>>(pool, table, ctx, (float*)rows, cu, B,
                                                            max_blocks, capacity, status);
  else
    gather_kernel<__nv_bfloat16><<<grid, kGatherThreads, smem, st>>>(
        pool, table, ctx, (__nv_bfloat16*)rows, cu, B, max_blocks, capacity, status);
  return cudaGetLastError();
}

}  // namespace mla
