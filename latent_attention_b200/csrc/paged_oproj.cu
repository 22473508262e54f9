// Output projection of the tensor-core paged decode: out = o W_o^T for the few
// rows of a decode batch, o as two bf16 terms (16 significant bits).
//
// The weights, [hidden, h dv], are read once and are what it takes; so they are
// the M side (128 rows of W_o a tile, the sequences as N: a product with the
// sequences as M would fill 128 rows whatever their number), and K is cut into
// enough pieces that every SM has some (a cluster of up to eight blocks a
// tile, whose fp32 sums are added up through distributed shared memory in a
// fixed order).  Both terms multiply a weight tile that stays in the collector.
// 96 rows, 4096 x 2048 weights (16.8 MB): 10 us, against 18 with the 256-column
// tiles of the large projections (16 blocks); bound by the launch and a few trips
// to memory.
#include <algorithm>

#include "ring_drain.cuh"
#include "sm100.cuh"
#include "tc.h"

namespace mla {
namespace {

using namespace sm100;

constexpr int NT = 128;
constexpr int ABOX = 128 * 128;          // 128 weight rows x 64 of K, bf16
constexpr int BN = 128;                  // sequences a block, at most
constexpr int MAX_STAGES = 10;           // 64 of K each, in 200 KB

struct OprojParams {
  __nv_bfloat16* out;                    // [B, hidden]
  int B, hidden, chunks;                 // K / 64, rounded up
  int bn;                                // sequences a block, multiple of 16
  int stages;
  uint32_t* status;
};
__host__ __device__ constexpr int stage_bytes(int bn) { return ABOX + 2 * bn * 128; }
// As deep a ring as fits: what streams is the weights, and four stages of them
// are too few in flight (16 sequences, 235 MB of weights: 64 us between events for
// 56; 4 sequences, 67 MB: 25.4 for 23.3).
int stages_of(int bn) { return std::min(MAX_STAGES, 200 * 1024 / stage_bytes(bn)); }
int smem_of(int bn) {
  // the ring, later the block's sums [bn][132]
  return std::max(stages_of(bn) * stage_bytes(bn), bn * 132 * 4) + 1024;
}

// Block (x, y, z): weight rows 128 x ..., piece y of K (the cluster), sequences
// bn z ...
__global__ void __launch_bounds__(NT) paged_oproj_kernel(const __grid_constant__ CUtensorMap tmW,
                                                         const __grid_constant__ CUtensorMap tmO,
                                                         const __grid_constant__ CUtensorMap tmL,
                                                         OprojParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[MAX_STAGES], empty[MAX_STAGES], done;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int n_pieces = gridDim.y, piece = blockIdx.y;
  const int n0 = blockIdx.x * 128, b0 = blockIdx.z * p.bn, nb = min(p.bn, p.B - b0);
  const int c0 = (int)((int64_t)p.chunks * piece / n_pieces);
  const int c1 = (int)((int64_t)p.chunks * (piece + 1) / n_pieces);
  const uint32_t cols = p.bn <= 32 ? 32 : p.bn <= 64 ? 64 : 128;
  if (t == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch(&tmW);
    tma_prefetch(&tmO);
    tma_prefetch(&tmL);
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, cols);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base;
  const int stage = stage_bytes(p.bn), stages = p.stages;
  // chunk i of the piece into slot s
  auto load_w = [&](int i, int s) {
    mbar_arrive_expect_tx(&full[s], stage);
    tma_load_2d(smem + s * stage, &tmW, (c0 + i) * 64, n0, &full[s]);
  };
  auto load_o = [&](int i, int s) {
    uint8_t* at = smem + s * stage + ABOX;
    tma_load_2d(at, &tmO, (c0 + i) * 64, b0, &full[s]);
    tma_load_2d(at + p.bn * 128, &tmL, (c0 + i) * 64, b0, &full[s]);
  };
  const int n = c1 - c0;
  volatile int* abort_v = &abort_flag;
  // the first weights do not depend on the kernel before this one (which
  // started only once all before it had finished)
  if (t == 32)
    for (int i = 0; i < min(n, stages); ++i) load_w(i, i);
  griddep_wait();
  griddep_launch_dependents();
  int issued = 0;                        // stages filled whole, by thread 32
  if (warp == 1) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0; i < n; ++i) {
        if (i >= stages) {
          if (!mbar_wait(&empty[s], ph, abort_v, p.status)) break;
          load_w(i, s);
        }
        load_o(i, s);
        issued = i + 1;
        if (++s == stages) { s = 0; ph ^= 1; }
      }
    }
  } else if (warp == 2) {
    if (elect_one()) {
      const uint32_t base = smem_u32(smem), idesc = idesc_bf16(128, p.bn);
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait(&full[s], ph, abort_v, p.status)) break;
        tc_fence_after();
        const uint32_t at = base + s * stage;
        const uint64_t da = desc_kmajor_sw128(at), dh = desc_kmajor_sw128(at + ABOX);
        const uint64_t dl = desc_kmajor_sw128(at + ABOX + p.bn * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mma_bf16_keep<false>(tbase, da + 2 * k, dh + 2 * k, idesc, (i | k) != 0);
          mma_bf16_keep<true>(tbase, da + 2 * k, dl + 2 * k, idesc, 1);
        }
        mma_commit(&empty[s]);
        if (++s == stages) { s = 0; ph ^= 1; }
      }
      mma_commit(&done);
    }
  }
  __syncwarp();
  // all threads: row n0 + t of the tile, into shared memory as [sequence][row]
  // (after a timeout the cluster goes on together; the status word says so)
  mbar_wait(&done, 0, abort_v, p.status);
  // a wait ran out somewhere: what is still in flight lands before the ring's
  // memory is the sums' (no weights are on their way alone: the first stages get
  // their o without a wait, the others both at once)
  if (t == 32 && *abort_v) {
    int given_up = 0;
    drain_ring(issued, stages, [](int) { return true; }, [&](int s, uint32_t parity) {
      mbar_wait(&full[s], parity, &given_up, nullptr);
    });
  }
  tc_fence_after();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
  for (int c = 0; c < p.bn; c += 16) {
    uint32_t v[16];
    tmem_ld16(tbase + ((uint32_t)(warp * 32) << 16) + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) sums[(c + k) * 132 + t] = __uint_as_float(v[k]);
  }
  tc_fence_before();
  cluster_sync_all();                    // the pieces' sums lie there
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tbase, cols);
  }
  // this block adds up every n_pieces-th sequence: a warp a row, a lane four of
  // its columns, the pieces in order
  for (int b = piece + n_pieces * warp; b < nb; b += n_pieces * 4) {
    const uint32_t at = smem_u32(sums + b * 132 + 4 * lane);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < n_pieces; ++q) {
      float4 x;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                   : "r"(mapa_shared(at, q))
                   : "memory");
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    const int col = n0 + 4 * lane;
    if (col < p.hidden)                  // hidden is a multiple of 8
      *reinterpret_cast<uint2*>(p.out + (int64_t)(b0 + b) * p.hidden + col) =
          make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
  cluster_sync_all();                    // read by all
}

}  // namespace

bool tc_paged_oproj_supported(const mla_config& c) { return c.hidden_size % 8 == 0; }

cudaError_t launch_paged_oproj(const void* o, const void* o_lo, const void* w_o, void* out, int B,
                               int K, int hidden, uint32_t* status, cudaStream_t st) {
  OprojParams p;
  p.out = (__nv_bfloat16*)out;
  p.B = B;
  p.hidden = hidden;
  p.chunks = (K + 63) / 64;
  p.bn = std::min(BN, (B + 15) / 16 * 16);
  p.stages = stages_of(p.bn);
  p.status = status;
  const int tiles = (hidden + 127) / 128, rows = (B + p.bn - 1) / p.bn;
  // pieces of K: blocks for every SM, eight chunks a piece at least
  int pieces = 1;
  while (pieces < 8 && 2 * pieces * tiles * rows <= kSMs && p.chunks >= 16 * pieces) pieces *= 2;
  CUtensorMap tmW, tmO, tmL;
  const uint64_t str[1] = {(uint64_t)K * 2};
  const uint64_t wd[2] = {(uint64_t)K, (uint64_t)hidden}, od[2] = {(uint64_t)K, (uint64_t)B};
  const uint32_t wb[2] = {64, 128}, ob[2] = {64, (uint32_t)p.bn};
  if (!encode_tmap(&tmW, w_o, 2, wd, str, wb) || !encode_tmap(&tmO, o, 2, od, str, ob) ||
      !encode_tmap(&tmL, o_lo, 2, od, str, ob))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> set{0};
  const cudaError_t e = set_dynamic_smem((const void*)paged_oproj_kernel, 201 * 1024, set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, pieces, rows);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem_of(p.bn);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.z = 1;
  attr[1].val.clusterDim.y = pieces;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches();
  return cudaLaunchKernelEx(&cfg, paged_oproj_kernel, tmW, tmO, tmL, p);
}

}  // namespace mla
