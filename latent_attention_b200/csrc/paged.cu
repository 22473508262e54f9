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
#include <algorithm>
#include <climits>

#include "paged.cuh"
#include "sm100.cuh"

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
// One block of 1024 threads computes the three prefix sums over the requests,
// a scan in registers and shared memory.  The entries that change hands and the
// slot map are spread flat over the threads (a binary search in a prefix finds
// an entry's request), so one long prompt costs no more than many short ones;
// many slots are left to a second grid, which finds the prefixes in the
// workspace.  A new token's block is looked up where it comes from, the old
// table or the ring, so nothing waits for the table to be written.
// All or nothing: if anything is out of range (a length, the ring's state, a
// block id that the step takes, gives back or fills further) or the ring or the
// slot map is too short, every output says "nothing happened".  So all ids are
// read before anything is written.
// It moves a few KB (a step of 256 requests) to some MB (prompts): a launch and
// three dependent trips to memory are its time, 5.7 us for a step of 256
// requests, 8.1 us for 61 prompts of 4000 tokens on average in blocks of 16 (1.6
// of it the look at 15000 ids by one block), 47 us for 8192 requests.

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

constexpr int kPlanThreads = 1024, kFillThreads = 256;
// One block writes up to this many slots itself (two rounds of its threads).
constexpr int kPlanOneBlock = 2048;

// What the entries and slots are found from, in shared memory or the workspace.
struct PlanSums {
  int32_t *add_end, *give_end, *new_end;   // [B] inclusive prefixes: blocks, blocks, tokens
  int32_t *held, *after;                   // [B] blocks before, tokens after the step
  int head, count, ta, tg, tn;             // ring before; blocks taken, given back; new tokens
};
__device__ __forceinline__ PlanSums sums_at(int32_t* base, int B) {
  PlanSums s;
  s.add_end = base; s.give_end = base + B; s.new_end = base + 2 * B;
  s.held = base + 3 * B; s.after = base + 4 * B;
  return s;
}

// (n_blocks is below 2^27: sums of two ring positions are ints)
__device__ __forceinline__ int wrap(int i, int n) { return i >= n ? i - n : i; }

// Entry i of the step's work: the i-th block taken, the i-th given back, the
// block and the position of the i-th new token; where each goes.
__device__ __forceinline__ int taken(const PlanArgs& a, const PlanSums& s, int i) {
  return a.ring[wrap(s.head + i, a.n_blocks)];
}
__device__ __forceinline__ void put_taken(const PlanArgs& a, const PlanSums& s, int i, int id) {
  const int b = request_of(s.add_end, a.B, i);
  a.table[(int64_t)b * a.max_blocks + s.held[b] + i - (b ? s.add_end[b - 1] : 0)] = id;
}
__device__ __forceinline__ int given(const PlanArgs& a, const PlanSums& s, int i) {
  const int b = request_of(s.give_end, a.B, i);
  return a.table[(int64_t)b * a.max_blocks + i - (b ? s.give_end[b - 1] : 0)];
}
__device__ __forceinline__ void put_given(const PlanArgs& a, const PlanSums& s, int i, int id) {
  a.ring[wrap(wrap(s.head + s.count, a.n_blocks) + i, a.n_blocks)] = id;
}
__device__ __forceinline__ int block_of(const PlanArgs& a, const PlanSums& s, int i, int& at) {
  const int b = request_of(s.new_end, a.B, i);
  at = s.after[b] - (s.new_end[b] - i);          // the request's last new token is after[b] - 1
  const int j = at / a.bs, had = s.held[b];
  return j < had ? a.table[(int64_t)b * a.max_blocks + j]
                 : taken(a, s, (b ? s.add_end[b - 1] : 0) + j - had);
}
__device__ __forceinline__ void put_slot(const PlanArgs& a, int i, int id, int at) {
  a.slots[i] = id < 0 ? -1 : id * a.bs + at % a.bs;
  if (a.pos) a.pos[i] = at;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a, int alone) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_sum[3][32];
  __shared__ int64_t totals[3];
  __shared__ int32_t s_head, s_count;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  PlanSums s = sums_at(sm, a.B);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    s_head = a.state[0];
    s_count = a.state[1];
    a.status[0] = a.status[1] = 0;
  }
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = t * per, b1 = min(b0 + per, a.B);
  const int lbs = __ffs(a.bs) - 1;
  int64_t add = 0, give = 0, fresh = 0;
  bool bad = false, bad_id = false;
  const auto look = [&](int id) { bad_id |= id < 0 || id >= a.n_blocks; };
  int part = 0;                                  // the id of a part-filled block that goes on
  for (int b = b0; b < b1; ++b) {
    const int64_t c = a.ctx[b], n = a.fresh[b];
    const int64_t grow = n > 0 ? n : 0;
    int64_t hb = (c + a.bs - 1) >> lbs, wb = (c + grow + a.bs - 1) >> lbs;
    if (c < 0 || n < -1 || wb > a.max_blocks) { bad = true; hb = wb = 0; }
    if (!alone) {                                // (used one request later, or behind the scan)
      look(part);
      part = n > 0 && hb > 0 && (c & (a.bs - 1)) ? a.table[(int64_t)b * a.max_blocks + hb - 1] : 0;
    }
    add += n < 0 ? 0 : wb - hb;
    give += n < 0 ? hb : 0;
    fresh += grow;
    s.held[b] = (int)hb;
    s.after[b] = n < 0 ? 0 : (int)(c + grow);
    // inclusive within this thread; the threads before it are added below
    s.add_end[b] = (int)add;
    s.give_end[b] = (int)give;
    s.new_end[b] = (int)fresh;
  }
  const int64_t ia = warp_scan(add, lane), ig = warp_scan(give, lane), in = warp_scan(fresh, lane);
  if (lane == 31) {
    warp_sum[0][warp] = ia;
    warp_sum[1][warp] = ig;
    warp_sum[2][warp] = in;
  }
  const int any_bad = __syncthreads_or(bad);
  if (warp < 3) {
    const int64_t v = warp_sum[warp][lane], x = warp_scan(v, lane);
    warp_sum[warp][lane] = x - v;
    if (lane == 31) totals[warp] = x;
  }
  __syncthreads();
  const int64_t ta = totals[0], tg = totals[1], tn = totals[2];
  const int n = a.n_blocks;
  s.head = s_head;
  s.count = s_count;
  const bool broken = any_bad || s.head < 0 || s.head >= n || s.count < 0 || s.count > n ||
                      s.count + tg > n;          // more blocks than the pool has
  const bool fits = !broken && ta <= s.count && tn <= a.capacity;
  s.ta = fits ? (int)ta : 0;
  s.tg = fits ? (int)tg : 0;
  s.tn = fits ? (int)tn : 0;
  // exclusive prefix of this thread's requests (int: used only when all fits)
  const int xa = (int)(warp_sum[0][warp] + ia - add), xg = (int)(warp_sum[1][warp] + ig - give),
            xn = (int)(warp_sum[2][warp] + in - fresh);
  for (int b = b0; b < b1; ++b) {
    s.add_end[b] += xa;
    s.give_end[b] += xg;
    s.new_end[b] += xn;
  }
  __syncthreads();
  // The ids of blocks that change hands or take new tokens.  A block alone keeps
  // what it read for the writes (kHeld entries of each kind a thread; every block
  // taken has a slot, so its id is looked at there).
  constexpr int kHeld = kPlanOneBlock / kPlanThreads;
  constexpr int kAsk = 8;                        // (16: the same; without: 8.9 us for the prompts)
  int id[kHeld], at[kHeld], take[kHeld], back[kHeld];
  if (alone) {
#pragma unroll
    for (int q = 0; q < kHeld; ++q) {
      const int i = t + q * kPlanThreads;
      id[q] = -1;
      at[q] = take[q] = back[q] = 0;
      if (i < s.ta) take[q] = taken(a, s, i);
      if (i < s.tn) look(id[q] = block_of(a, s, i, at[q]));
      if (i < s.tg) look(back[q] = given(a, s, i));
    }
    for (int i = t + kHeld * kPlanThreads; i < s.tg; i += kPlanThreads) look(given(a, s, i));
  } else {
    look(part);
    for (int i = t; i < s.ta; i += kAsk * kPlanThreads) {
      int v[kAsk];
#pragma unroll
      for (int q = 0; q < kAsk; ++q)
        v[q] = i + q * kPlanThreads < s.ta ? taken(a, s, i + q * kPlanThreads) : 0;
#pragma unroll
      for (int q = 0; q < kAsk; ++q) look(v[q]);
    }
    for (int i = t; i < s.tg; i += kPlanThreads) look(given(a, s, i));
  }
  const bool broken_id = __syncthreads_or(bad_id) && fits, ok = fits && !broken_id;
  if (!ok) s.ta = s.tg = s.tn = 0;
  for (int b = b0; b < b1; ++b) {
    a.cu[b + 1] = ok ? s.new_end[b] : 0;
    const int32_t was = a.ctx[b];                // before ctx_out, which may be ctx
    a.ctx_out[b] = ok ? s.after[b] : was;
  }
  if (t == 0) {
    a.cu[0] = 0;
    a.state_out[0] = ok ? wrap(s.head + (int)ta, n) : s.head;
    a.state_out[1] = ok ? (int)(s.count - ta + tg) : s.count;
    if (!ok) atomicOr(a.status, broken || broken_id ? kStatusBadPage : kStatusNoBlocks);
    if (!alone) {
      a.sums[0] = s.head; a.sums[1] = s.count; a.sums[2] = s.ta; a.sums[3] = s.tg;
      a.sums[4] = s.tn;
    }
  }
  if (!alone) {
    for (int i = t; i < 5 * a.B; i += kPlanThreads) a.sums[8 + i] = sm[i];
    return;
  }
#pragma unroll
  for (int q = 0; q < kHeld; ++q) {
    const int i = t + q * kPlanThreads;
    if (i < s.ta) put_taken(a, s, i, take[q]);
    if (i < s.tg) put_given(a, s, i, back[q]);
    if (i < a.capacity) put_slot(a, i, ok ? id[q] : -1, ok ? at[q] : 0);
  }
  for (int i = t + kHeld * kPlanThreads; i < s.tg; i += kPlanThreads)
    put_given(a, s, i, given(a, s, i));
}

// Entries and slots on their own grid; the ids have been checked.
__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(PlanArgs a) {
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  PlanSums s = sums_at(a.sums + 8, a.B);
  s.head = a.sums[0]; s.count = a.sums[1]; s.ta = a.sums[2]; s.tg = a.sums[3]; s.tn = a.sums[4];
  const int first = blockIdx.x * kFillThreads + threadIdx.x, step = gridDim.x * kFillThreads;
  for (int i = first; i < s.ta; i += step) put_taken(a, s, i, taken(a, s, i));
  for (int i = first; i < s.tg; i += step) put_given(a, s, i, given(a, s, i));
  for (int i = first; i < a.capacity; i += step) {
    int id = -1, at = 0;
    if (i < s.tn) id = block_of(a, s, i, at);
    put_slot(a, i, id, at);
  }
}

// ----------------------------------------------------------------- append
//
// A run is a maximal stretch of rows whose slots are consecutive in one
// block; one CTA quantises it:  e = min{e : max|row| <= 448 2^e}; rows of the
// block in front of the run (offsets below its first slot) are kept and moved
// to max(e, e_old).  Rows behind the run are dead and stay as they were.
// A CTA takes the runs that start in its window of the slot map.  A run's values
// stay in registers between the maximum and the rounding (the first HELD pieces
// of 16 a thread; the rest of a longer run is read again).  Where a window of
// a 1024-thread block holds more than two runs, those of up to kShortRun rows
// take a warp each and go side by side (the new tokens of many requests); the
// others take the whole block.  (256-thread blocks do without: the mere code
// cost 48624 rows in 1500 runs 4 us of 23.)  What bounds it is trips to memory
// (slots, rows, the block's claim, then the writes) with few instructions a
// value: maxima of two bf16 at a time as integers, packed products, 16 bytes a
// store.  48624 rows, 84 MB: 18.8 us with the rows in L2 (22.8 with a maximum and
// a test for infinities per value), 24.6 from memory, 3.4 TB/s.

// A block's status at its end (of all threads, after a barrier): a word of its
// own, or into the status word that was cleared before the launch.
__device__ __forceinline__ void report(uint32_t* status, uint32_t flags, bool own) {
  if (threadIdx.x != 0) return;
  if (own) {
    status[kStatusSlots + blockIdx.x] = flags;
    if (blockIdx.x == 0) {
      status[0] = 0;
      status[1] = kStatusMagic + gridDim.x;
    }
  } else if (flags) {
    atomicOr(status, flags);
  }
}

// (500 runs of 6 rows: 9.1 us, 14.9 with the limit at 4; at 16, 195 runs of 26
// rows, cut by blocks of 64, take 14.5 us for 12.5.)
constexpr int kShortRun = 8;

// Largest |x| of a piece as bits, NaN and infinity above all numbers.
__device__ __forceinline__ uint32_t largest(const Piece<float>& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, x.w[i] & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t largest(const Piece<__nv_bfloat16>& x) {
  uint32_t m = 0;                            // two at a time: their bits are 16-bit integers
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_u16x2(m, x.w[i] & 0x7fff7fffu);
  return max(m << 16, m & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ void maxima(const Piece<T>& x, uint32_t& amax, uint32_t& odd) {
  const uint32_t m = largest(x);
  if (m < 0x7f800000u) {
    amax = max(amax, m);
    return;
  }
  float v[16];
  values(x, v);
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    const uint32_t b = __float_as_uint(v[y]) & 0x7fffffffu;
    if (b < 0x7f800000u) amax = max(amax, b); else odd = 1;
  }
}
__device__ __forceinline__ uint4 to_bytes(const float (&v)[16]) {
  return make_uint4(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]),
                    to_e4m3x4(v[8], v[9], v[10], v[11]), to_e4m3x4(v[12], v[13], v[14], v[15]));
}

// One run by G threads (a warp or the block).  share(amax, odd, refused) makes
// the three values those of all threads; odd: any NaN or infinity.
template <typename T, int G, int HELD, typename Share>
__device__ __forceinline__ void append_run(const T* __restrict__ rows,
                                           const int32_t* __restrict__ slots, const PagedPool& pool,
                                           int i, int s, int len, int t, bool wide,
                                           uint32_t* claims, uint32_t* flags, Share share) {
  const int W = pool.W, bs = pool.bs, blk = s / bs, off = s % bs, nv = len * W / 16;
  const T* src = rows + (int64_t)i * W;
  Piece<T> held[HELD];
#pragma unroll
  for (int q = 0; q < HELD; ++q)
    if (t + q * G < nv) load_piece(src + (t + q * G) * 16, wide, held[q]);
  // two runs of one call in one block have no order: the second is refused
  uint32_t refused = 0;
  if (G == 256 || claims) {                  // (256 threads: many rows, always by claims)
    const uint32_t bit = 1u << (blk & 31);
    if (t == 0 && (atomicOr(&claims[blk >> 5], bit) & bit)) refused = 1;
  } else {
    const int lbs = __ffs(bs) - 1;           // (a negative slot stays negative)
#pragma unroll 8
    for (int q = t; q < i; q += G) refused |= slots[q] >> lbs == blk;
  }
  const float old_scale = off > 0 ? pool.scales[blk] : 1.f;
  uint32_t amax = 0, odd = 0;
#pragma unroll
  for (int q = 0; q < HELD; ++q)
    if (t + q * G < nv) maxima(held[q], amax, odd);
  for (int p = t + HELD * G; p < nv; p += G) {
    Piece<T> x;
    load_piece(src + p * 16, wide, x);
    maxima(x, amax, odd);
  }
  share(amax, odd, refused);
  if (refused) {
    if (t == 0) atomicOr(flags, kStatusBadPage);
    return;
  }
  int e = scale_exp(amax), e_old = e;
  uint8_t* base = pool.cache + (int64_t)blk * bs * W;
  if (off > 0) {
    if (stored_exp(old_scale, &e_old)) {
      e = max(e, e_old);
    } else {
      if (t == 0) atomicOr(flags, kStatusBadPage);
      e_old = e;
    }
  }
  if (e != e_old) {                          // the kept rows move to the larger scale
    const float f = pow2(e_old - e);
    uint4* kept = reinterpret_cast<uint4*>(base);
#pragma unroll 4
    for (int p = t; p < off * W / 16; p += G) {
      float v[16];
      dequant16(kept[p], f, v);
      kept[p] = to_bytes(v);
    }
  }
  const float f = pow2(-e);
  uint4* dst = reinterpret_cast<uint4*>(base + (int64_t)off * W);
  auto put = [&](int p, const Piece<T>& x) {
    float v[16];
    values(x, v);
    if (odd) {                               // an infinity is stored as NaN, not 448
#pragma unroll
      for (int y = 0; y < 16; ++y) v[y] += v[y] - v[y];
    }
#pragma unroll
    for (int y = 0; y < 16; y += 2) mul2(v[y], v[y + 1], f, f);
    dst[p] = to_bytes(v);
  };
#pragma unroll
  for (int q = 0; q < HELD; ++q)
    if (t + q * G < nv) put(t + q * G, held[q]);
  for (int p = t + HELD * G; p < nv; p += G) {
    Piece<T> x;
    load_piece(src + p * 16, wide, x);
    put(p, x);
  }
  if (t == 0) pool.scales[blk] = pow2(e);    // (every thread has read it: share)
}

// (fp32 pieces take twice the registers; held to four blocks an SM all the same,
// 48624 rows took 14.5 us instead of 18.6, while bf16's third block to a fourth
// gains nothing.)
template <typename T, int NT>
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : sizeof(T) == 4 ? 4 : 3)
    append_kernel(const T* __restrict__ rows, const int32_t* __restrict__ slots, int n_rows,
                  PagedPool pool, int window, uint32_t* status, uint32_t* claims) {
  constexpr int HELD = NT == 256 ? 5 : sizeof(T) == 2 ? 3 : 2;
  __shared__ int sl[258];                   // slots w0 - 1 .. w1 + bs - 1
  __shared__ int starts[128], lens[128], n_starts, run_len;
  __shared__ uint32_t s_val[3], flags;      // a run's maximum, odd, refused; this block's status
  const int t = threadIdx.x, bs = pool.bs;
  const int64_t n_slots = (int64_t)pool.n_blocks * bs;
  const bool wide = aligned32(rows);        // rows are a multiple of 32 bytes
  const int w0 = blockIdx.x * window, w1 = min(w0 + window, n_rows);
  if (t == 0) {
    n_starts = 0;
    flags = 0;
    // the rows do not wait for the slots: from memory, 65536 rows take 31 us
    // instead of 37, and 48624 24.6 instead of 26.6
    if (NT == 256)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(rows + (int64_t)w0 * pool.W),
                   "r"((w1 - w0) * pool.W * (int)sizeof(T))
                   : "memory");
  }
  for (int k = t; k < w1 - w0 + bs + 1; k += NT) {
    const int i = w0 - 1 + k;
    sl[k] = i >= 0 && i < n_rows ? slots[i] : -1;
  }
  __syncthreads();
  if (t < w1 - w0) {
    const int s = sl[t + 1], before = sl[t];
    const bool in = s >= 0 && s < n_slots;
    // a row of the block that the row before it writes: part of that run, or
    // (not its next slot) refused
    const bool cont = in && before >= 0 && before / bs == s / bs;
    if ((!in && s != -1) || (cont && before + 1 != s)) atomicOr(&flags, kStatusBadPage);
    if (in && !cont) {
      const int k = atomicAdd(&n_starts, 1), most = min(bs - s % bs, n_rows - w0 - t);
      int len = 1;                          // up to kShortRun + 1
      while (len <= kShortRun && len < most && sl[t + 1 + len] == s + len) ++len;
      starts[k] = w0 + t;
      lens[k] = len;
    }
  }
  __syncthreads();
  const int todo = n_starts;
  const bool apart = NT == 1024 && todo > 2;
  if constexpr (NT == 1024) {
    for (int k = t / 32; apart && k < todo; k += NT / 32)
      if (lens[k] <= kShortRun)
        append_run<T, 32, sizeof(T) == 2 ? 4 : 2>(
            rows, slots, pool, starts[k], sl[starts[k] - w0 + 1], lens[k], t & 31, wide, claims,
            &flags, [](uint32_t& amax, uint32_t& odd, uint32_t& refused) {
              amax = __reduce_max_sync(0xffffffffu, amax);
              odd = __reduce_or_sync(0xffffffffu, odd);
              refused = __reduce_or_sync(0xffffffffu, refused);
            });
  }
  for (int k = 0; k < todo; ++k) {
    if (apart && lens[k] <= kShortRun) continue;
    const int i = starts[k], s = sl[i - w0 + 1];
    const int most = min(bs - s % bs, n_rows - i);
    __syncthreads();                        // the run before is done with the shared values
    if (t == 0) {
      run_len = most;
      s_val[0] = s_val[1] = s_val[2] = 0;
    }
    __syncthreads();
    if (t < most && sl[i - w0 + 1 + t] != s + t) atomicMin(&run_len, t);
    __syncthreads();
    append_run<T, NT, HELD>(rows, slots, pool, i, s, run_len, t, wide, claims, &flags,
                            [&](uint32_t& amax, uint32_t& odd, uint32_t& refused) {
                              amax = __reduce_max_sync(0xffffffffu, amax);
                              odd = __reduce_or_sync(0xffffffffu, odd);
                              refused = __reduce_or_sync(0xffffffffu, refused);
                              if ((t & 31) == 0) {
                                atomicMax(&s_val[0], amax);
                                if (odd) atomicOr(&s_val[1], 1u);
                                if (refused) atomicOr(&s_val[2], 1u);
                              }
                              __syncthreads();
                              amax = s_val[0];
                              odd = s_val[1];
                              refused = s_val[2];
                            });
  }
  __syncthreads();
  report(status, flags, NT == 1024 && !claims);
}

// ----------------------------------------------------------------- gather
//
// Rows of all requests back to back, and their prefix sums.  Each CTA scans
// the lengths into shared memory and takes tiles of kGatherRows rows: the
// tile's source rows are looked up once, then a thread takes one 16-byte
// column of every R-th row, four loads in flight.  Memory bounds it (1152 bytes
// written and 576 read a token in bf16): 556900 tokens, 0.96 GB, take 164 us, 5.9
// TB/s; 8192 tokens 4.8 us, where looking up rows before bytes is two trips.
constexpr int kGatherThreads = 288, kGatherRows = 32, kGatherFly = 4;

template <typename T>
__global__ void __launch_bounds__(kGatherThreads)
    gather_kernel(PagedPool pool, const int32_t* __restrict__ table,
                  const int32_t* __restrict__ ctx, T* __restrict__ rows, int32_t* __restrict__ cu,
                  int B, int max_blocks, int capacity, uint32_t* status) {
  extern __shared__ int32_t ends[];          // [B] inclusive prefix sums
  __shared__ int64_t warp_sum[kGatherThreads / 32];
  __shared__ int64_t src[2][kGatherRows];    // byte offset of a tile's rows, or -1
  __shared__ float scl[2][kGatherRows];
  __shared__ uint32_t flags;                 // this block's status
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) flags = 0;
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
    if (bad || (t == 0 && total > capacity)) atomicOr(&flags, kStatusBadPage);
    if (t == 0) cu[0] = 0;
  }
  const int n_rows = min(total, capacity), nv = pool.W / 16;
  // threads of a row, rows at a time; wide rows take several rounds of columns
  const int tv = min(nv, kGatherThreads), R = kGatherThreads / tv;
  const int c0 = t % tv, r0 = t / tv;
  const bool wide = aligned32(rows);
  auto look_up = [&](int first, int buf) {
    if (t < kGatherRows) {
      int64_t o = -1;
      float s = 0.f;
      const int i = first + t;
      if (i < n_rows) {
        const int b = request_of(ends, B, i);
        const int j = i - (b ? ends[b - 1] : 0);
        const int blk = table[(int64_t)b * max_blocks + j / pool.bs];
        if (blk >= 0 && blk < pool.n_blocks) {
          o = ((int64_t)blk * pool.bs + j % pool.bs) * pool.W;
          s = read_scale(pool.scales[blk], &flags);
        } else {
          atomicOr(&flags, kStatusBadPage);
        }
      }
      src[buf][t] = o;
      scl[buf][t] = s;
    }
  };
  const int stride = gridDim.x * kGatherRows;
  int buf = 0;
  if (blockIdx.x * kGatherRows < n_rows) look_up(blockIdx.x * kGatherRows, 0);
  for (int first = blockIdx.x * kGatherRows; first < n_rows; first += stride, buf ^= 1) {
    __syncthreads();                         // the tile's rows are known
    if (first + stride < n_rows) look_up(first + stride, buf ^ 1);
    const int here = min(kGatherRows, n_rows - first);
    if (r0 < R) {
      for (int c = c0; c < nv; c += tv) {
        for (int rb = r0; rb < here; rb += R * kGatherFly) {
          uint4 x[kGatherFly];
#pragma unroll
          for (int q = 0; q < kGatherFly; ++q) {
            const int r = rb + q * R;
            x[q] = make_uint4(0u, 0u, 0u, 0u);   // a row whose block is out of range
            if (r < here && src[buf][r] >= 0)
              x[q] = *reinterpret_cast<const uint4*>(pool.cache + src[buf][r] + c * 16);
          }
#pragma unroll
          for (int q = 0; q < kGatherFly; ++q) {
            const int r = rb + q * R;
            if (r >= here) break;
            float v[16];
            Piece<T> out;
            dequant16(x[q], scl[buf][r], v);
            piece_of(v, out);
            store_piece(rows + (int64_t)(first + r) * pool.W + c * 16, wide, out);
          }
        }
      }
    }
  }
  __syncthreads();
  report(status, flags, true);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)plan_kernel, 5 * 4 * kMaxRequests, set);
  if (e != cudaSuccess) return e;
  const bool alone = a.capacity <= kPlanOneBlock;
  const cudaError_t e1 = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads),
                                    5 * 4 * (size_t)a.B, st, a, (int)alone);
  count_launches();
  if (e1 != cudaSuccess || alone) return e1;
  const int grid = std::min((a.capacity + kFillThreads - 1) / kFillThreads, 8 * kSMs);
  count_launches();
  return launch_pdl(plan_fill_kernel, dim3(grid), dim3(kFillThreads), 0, st, a);
}

cudaError_t launch_paged_append(int dtype, const void* rows, const int32_t* slots, int n_rows,
                                const PagedPool& pool, uint32_t* status, uint32_t* claims,
                                cudaStream_t st) {
  // Fewer runs of whole blocks than twice the SMs: blocks of 1024 threads, one an
  // SM (4096 rows in 64 runs 6.2 us, against 10.2 with four windows an SM, whose
  // empty blocks are in the way, and 11.0 with 256 threads).  Beyond: 256 threads
  // and four windows an SM, whose blocks overlap each other's trips to memory.
  const bool few = n_rows < 2 * kSMs * pool.bs;
  const int windows = few ? kSMs : 4 * kSMs;
  const int window = std::min((n_rows + windows - 1) / windows, pool.bs);
  const int grid = (n_rows + window - 1) / window;
  static_assert(kAppendScan < 2 * kSMs * 16, "256-thread blocks take claims");
  if (n_rows <= kAppendScan) claims = nullptr;   // (at most 4096 / 16 blocks)
  count_launches();
  const auto go = [&](auto kernel, auto* p, int nt) {
    kernel<<<grid, nt, 0, st>>>(p, slots, n_rows, pool, window, status, claims);
  };
  if (dtype == MLA_F32) {
    if (few) go(append_kernel<float, 1024>, (const float*)rows, 1024);
    else go(append_kernel<float, 256>, (const float*)rows, 256);
  } else {
    const auto* p = (const __nv_bfloat16*)rows;
    if (few) go(append_kernel<__nv_bfloat16, 1024>, p, 1024);
    else go(append_kernel<__nv_bfloat16, 256>, p, 256);
  }
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(int dtype, const PagedPool& pool, const int32_t* table,
                                const int32_t* ctx, void* rows, int32_t* cu, int B,
                                int max_blocks, int capacity, uint32_t* status, cudaStream_t st) {
  const int tiles = (capacity + kGatherRows - 1) / kGatherRows;
  const int grid = tiles < 8 * kSMs ? (tiles > 0 ? tiles : 1) : 8 * kSMs;
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
