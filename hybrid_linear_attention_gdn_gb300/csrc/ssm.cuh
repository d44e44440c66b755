// Selective state space step: pieces shared by its kernels.
#pragma once
#include "gdn_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kMaxW = 8;

// dt = softplus(a + dt_bias) and the log decay -exp(A_log) dt of a token
struct Gate {
  float dt, g;
};
__device__ __forceinline__ Gate gate(float A_log, float dt_bias, float a) {
  Gate r;
  r.dt = softplus_f(a + dt_bias);
  r.g = -expf(A_log) * r.dt;
  return r;
}

// Kernel K's dynamic shared memory limit, raised on its first launch on a
// device (`bytes` the same on every call).  Threads that come first together
// each raise it.
template <auto K>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<bool> done[64];
  int dev = 0;
  const cudaError_t d = cudaGetDevice(&dev);
  if (d != cudaSuccess) return d;
  const bool known = dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (known && e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

struct DecodeArgs {
  float* ssm;
  void* conv;
  int32_t num_slots;
  const float* conv_w;
  const float* conv_bias;
  const float* A_log;
  const float* dt_bias;
  const float* D;
  const int32_t* slot_ids;
  int32_t B;
  const void* qkv;
  const void* a;
  void* out;
  uint32_t* err;
  int32_t hk, hv, dv, W, C, G;
  int32_t cs, rpc;  // CTAs per (request, QK head); rows per CTA
};

// the persistent form for large batches (ssm_ring.cu)
bool decode_ring_supported(const gdn_dims& d, int32_t B, const void* qkv, const gdn_ssm_params& p);
cudaError_t decode_ring_launch(const DecodeArgs& a, int act, int cv, cudaStream_t s);

struct PrefillArgs {
  float* ssm;
  const void* conv;
  int32_t num_slots;
  float* ck_ssm;
  int32_t ck_num_slots;
  const float* conv_w;
  const float* conv_bias;
  const float* A_log;
  const float* dt_bias;
  const float* D;
  const int32_t* slot_ids;
  const int32_t* cu_seqlens;
  const int64_t* start_pos;
  int32_t n_seq;
  int64_t total;
  const int32_t* ckpt_ids;
  int32_t max_ckpt;
  int32_t ckpt_block;
  const void* qkv;
  const void* a;
  void* out;
  uint32_t* err;
  int32_t hk, hv, dk, dv, W, C, G;
};

}  // namespace ssm
}  // namespace gdn
