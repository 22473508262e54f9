// Tensor-core (tcgen05 / TMEM / TMA) path for sm_100a, bf16 operands.
#pragma once
#include "internal.h"

namespace mla {

// Column tile width of the tensor-core GEMM.
constexpr int kTcTileN = 256;

// Whether the tensor-core attention kernel takes this configuration.
bool tc_attention_supported(const mla_config& c);
// Whether a single GEMM can run on the tensor-core kernel.
bool tc_gemm_supported(const GemmArgs& a, int dtype);
cudaError_t tc_gemm(const GemmArgs& a, cudaStream_t st, uint32_t* status);
cudaError_t tc_attention(const AttnArgs& a, cudaStream_t st);
bool tc_decode_supported(const mla_config& c);
cudaError_t tc_decode(const DecodeArgs& a, cudaStream_t st);
// Shortest slice of the token stream one CTA pair of the tensor-core decode
// takes (tokens).
int tc_decode_min_slice();
// The paged decode's tensor-core kernel: the shapes it takes, how it divides
// h heads over `sms` SMs.
bool tc_paged_supported(const mla_config& c);
PagedTcPlan tc_paged_plan(int h, int sms);
cudaError_t tc_paged_decode(const PagedDecodeArgs& a, cudaStream_t st);
// Its projections: query (and lengths, status word), output.
cudaError_t launch_paged_query(const PagedDecodeArgs& a, int min_len, cudaStream_t st);
cudaError_t launch_paged_output(const PagedDecodeArgs& a, cudaStream_t st);
// out [B, hidden] = (o + o_lo) [B, K] w_o [hidden, K]^T.
bool tc_paged_oproj_supported(const mla_config& c);
cudaError_t launch_paged_oproj(const void* o, const void* o_lo, const void* w_o, void* out, int B,
                               int K, int hidden, uint32_t* status, cudaStream_t st);

}  // namespace mla
