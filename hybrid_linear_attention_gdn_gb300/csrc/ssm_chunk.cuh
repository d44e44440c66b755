// Chunked prefill of the selective state space step (ssm_chunk.cu).
#pragma once
#include "ssm.cuh"

namespace gdn {
// whether dims take the chunked form, and whether a call's tensors and sizes do
bool ssm_chunk_shape(const gdn_dims& d);
bool ssm_chunk_supported(const gdn_dims& d, int32_t n_seq, int64_t total, const void* qkv, const void* out,
                         const gdn_ssm_params& p);
size_t ssm_chunk_workspace(const gdn_dims& d, int32_t n_seq, int64_t total);
// the whole prefill: outputs, states, checkpoints and conv histories
cudaError_t ssm_chunk_launch(const ssm::PrefillArgs& p, const gdn_dims& d, void* ck_conv, void* workspace,
                             cudaStream_t s);
}  // namespace gdn
