// Residual addition and RMS norm between the layers, with an e4m3 output and
// its scales for the next projection.
//
// Not written on the pages; the published pre-norm block:
//   h = x + residual;  residual <- h;  y = h / sqrt(mean(h^2) + eps) * weight
// and q8 = y / scale with one scale per group of consecutive values (or per
// row), scale = max|y| / 448 in fp32 or the next power of two.
//
// HBM bound: x and the residual are read once, the residual, y and q8
// written once; h stays in registers between the sum of squares and the
// outputs.  A row belongs to TPR threads, thread t of a row holding the V
// vectors of 8 consecutive values from 8 (v TPR + t): a vector is one or two
// 16-byte accesses, consecutive threads touch consecutive vectors, and a
// scale group of 32 .. 256 values is 4 .. 32 neighbouring lanes, reduced by
// shuffles.  TPR is the smallest of 32 .. 1024 threads that needs at most
// four vectors (d up to 32768), and rows shorter than 256 threads' worth
// share a CTA, so that short and long rows alike keep about 2,000 threads
// with loads in flight on every SM.  The same code with element accesses
// takes any alignment and any d.
//
// Measured: 32768 rows of 4096, bf16 with an fp32 residual, y and q8: 248 us,
// 1.04 of the copy bandwidth (1.75 GB); 64 rows 3.5 us in a graph of calls.
#include "gdn_common.cuh"

#include <cuda_fp8.h>

namespace gdn {
namespace {

struct NormArgs {
  const void* x;
  void* residual;
  const float* weight;
  float eps;
  int64_t n_rows;
  int32_t d;
  void* y;
  uint8_t* q8;
  void* scales;
  int32_t group, scale_type;
};

// 8 consecutive elements from p[0], as fp32; VEC: p is 16-byte aligned and
// all 8 exist, else the first n of them (the others 0)
template <bool VEC, typename T, typename VT>
__device__ __forceinline__ void load8(float (&f)[8], const VT& p, int64_t at, int n) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? to_f32(p[at + i]) : 0.f;
  } else if constexpr (sizeof(T) == 4) {
    const float4 u = vec_at<const float4>(p, at), v = vec_at<const float4>(p, at + 4);
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
    f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
  } else {
    const uint4 u = vec_at<const uint4>(p, at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}
template <bool VEC, typename T, typename VT>
__device__ __forceinline__ void store8(const float (&f)[8], const VT& p, int64_t at, int n) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[at + i] = from_f32<T>(f[i]);
  } else if constexpr (sizeof(T) == 4) {
    vec_at<float4>(p, at) = make_float4(f[0], f[1], f[2], f[3]);
    vec_at<float4>(p, at + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint4 u;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    u.x = w[0]; u.y = w[1]; u.z = w[2]; u.w = w[3];
    vec_at<uint4>(p, at) = u;
  }
}

// the larger of two magnitudes, NaN if either is (fmaxf would drop it)
__device__ __forceinline__ float amax2(float a, float b) { return (a > b || a != a) ? a : b; }

// the scale of a group whose largest |y| is m, stored at index `at`; returns
// 1 / scale (0 only for an infinite scale).  e4m3's largest value is 448.
__device__ __forceinline__ float put_scale(const NormArgs& a, float m, int64_t at, int64_t n_scales, bool store) {
  if (a.scale_type == GDN_SCALE_F32) {
    // at least 2^-126: a smaller scale's reciprocal could overflow
    float s = m == 0.f ? 1.f : m / 448.f;
    s = s < 1.17549435e-38f ? 1.17549435e-38f : s;
    if (store) GDN_GV(reinterpret_cast<float*>(a.scales), n_scales)[at] = s;
    return 1.f / s;
  }
  // byte b stands for 2^(b - 127): the smallest with 448 * 2^(b - 127) >= m
  int b = 127;
  if (m != m) {
    b = 255;
  } else if (m > 0.f) {
    const float s = m / 448.f;
    const uint32_t u = __float_as_uint(s);
    // the exponent, rounded up; byte 0 is the subnormal 2^-127
    b = u > 0x400000u ? (int)(u >> 23) + ((u & 0x7fffffu) ? 1 : 0) : 0;
    // the division may have rounded down onto a power of two below m / 448
    if (b < 254 && b > 0 && 448.f * __uint_as_float((uint32_t)b << 23) < m) ++b;
    b = b > 254 ? 254 : b;
  }
  if (store) GDN_GV(reinterpret_cast<uint8_t*>(a.scales), n_scales)[at] = (uint8_t)b;
  if (b == 255) return __uint_as_float(0x7fc00000u);
  // 2^(127 - b) as a float: normal for b <= 253, subnormal for 254
  return b < 254 ? __uint_as_float((uint32_t)(254 - b) << 23) : 5.87747175e-39f;
}

// TPR threads per row, ROWS rows per CTA
template <typename Tact, typename Tres, int TPR, int ROWS, int V, bool VEC>
__global__ void __launch_bounds__(TPR* ROWS) add_rmsnorm_kernel(const NormArgs a) {
  constexpr int kRowWarps = TPR / 32;
  __shared__ float red[ROWS][32];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x % TPR, rloc = threadIdx.x / TPR, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * ROWS + rloc;
  const bool live = row < a.n_rows;  // the same for the threads of a row
  const int64_t n = a.n_rows * a.d, base = row * a.d;
  const auto x = GDN_GV(reinterpret_cast<const Tact*>(a.x), n);
  const auto res = GDN_GV(reinterpret_cast<Tres*>(a.residual), n);
  const auto w = GDN_GV(a.weight, a.d);
  float h[V][8];
  float ss = 0.f;
  if (live) {
    float r[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * TPR + t);
      if (c < a.d) {
        load8<VEC, Tact>(h[v], x, base + c, a.d - c);
        if (a.residual) load8<VEC, Tres>(r[v], res, base + c, a.d - c);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * TPR + t);
      if (c < a.d) {
        if (a.residual) {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] += r[v][i];
          store8<VEC, Tres>(h[v], res, base + c, a.d - c);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (kRowWarps > 1) {
    if (lane == 0) red[rloc][t >> 5] = ss;
    __syncthreads();
    ss = lane < kRowWarps ? red[rloc][lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float inv = 1.f / sqrtf(ss / (float)a.d + a.eps);
  float top = 0.f;  // the row's largest |y| (one scale per row)
  if (live) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * TPR + t);
      if (c < a.d) {
        float g[8];
        load8<VEC, float>(g, w, c, a.d - c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[v][i] = h[v][i] * inv * g[i];
          top = amax2(fabsf(h[v][i]), top);
        }
        if (a.y) store8<VEC, Tact>(h[v], GDN_GV(reinterpret_cast<Tact*>(a.y), n), base + c, a.d - c);
      }
    }
  }
  if (!a.q8) return;
  const int64_t per_row = a.group ? a.d / a.group : 1, n_scales = a.n_rows * per_row;
  float scale_inv = 0.f;
  if (a.group == 0) {
#pragma unroll
    for (int o = 16; o; o >>= 1) top = amax2(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (kRowWarps > 1) {
      __syncthreads();  // red has been read
      if (lane == 0) red[rloc][t >> 5] = top;
      __syncthreads();
      top = lane < kRowWarps ? red[rloc][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = amax2(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (live) scale_inv = put_scale(a, top, row, n_scales, t == 0);
  }
  const auto q8 = GDN_GV(a.q8, n);
  const int gl = a.group / 8;  // lanes of a group
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * TPR + t);
    const bool in = live && c < a.d;
    float inv_s = scale_inv;
    if (a.group) {
      float m = 0.f;
      if (in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = amax2(fabsf(h[v][i]), m);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, m, o);
        if (o < gl) m = amax2(m, u);
      }
      if (in) inv_s = put_scale(a, m, row * per_row + c / a.group, n_scales, t % gl == 0);
    }
    if (!in) continue;
    uint32_t q[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = make_float2(h[v][2 * i] * inv_s, h[v][2 * i + 1] * inv_s);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3);
      q[i >> 1] |= b << (16 * (i & 1));
    }
    if constexpr (VEC) {
      vec_at<uint2>(q8, base + c) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < a.d - c) q8[base + c + i] = (uint8_t)(q[i >> 2] >> (8 * (i & 3)));
    }
  }
}

template <typename Tact, typename Tres, int TPR, int ROWS, int V>
cudaError_t launch_norm(const NormArgs& a, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)((a.n_rows + ROWS - 1) / ROWS)), block(TPR * ROWS);
  return vec ? launch_pdl(add_rmsnorm_kernel<Tact, Tres, TPR, ROWS, V, true>, grid, block, 0, s, dim3(1), a)
             : launch_pdl(add_rmsnorm_kernel<Tact, Tres, TPR, ROWS, V, false>, grid, block, 0, s, dim3(1), a);
}

template <typename Tact, typename Tres>
cudaError_t dispatch_norm(const NormArgs& a, bool vec, cudaStream_t s) {
  if (a.d <= 256) return launch_norm<Tact, Tres, 32, 8, 1>(a, vec, s);
  if (a.d <= 1024) return launch_norm<Tact, Tres, 128, 2, 1>(a, vec, s);
  if (a.d <= 2048) return launch_norm<Tact, Tres, 256, 1, 1>(a, vec, s);
  if (a.d <= 4096) return launch_norm<Tact, Tres, 256, 1, 2>(a, vec, s);
  if (a.d <= 8192) return launch_norm<Tact, Tres, 512, 1, 2>(a, vec, s);
  if (a.d <= 16384) return launch_norm<Tact, Tres, 1024, 1, 2>(a, vec, s);
  return launch_norm<Tact, Tres, 1024, 1, 4>(a, vec, s);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_add_rmsnorm(int32_t act_dtype, int32_t res_dtype, const void* x, void* residual,
                                      const float* weight, float eps, int64_t n_rows, int32_t d, void* y, void* q8,
                                      void* scales, int32_t group, int32_t scale_type, void* stream) {
  using namespace gdn;
  if (act_dtype != GDN_F32 && act_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (res_dtype != GDN_F32 && res_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (n_rows < 0 || d <= 0 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256) return GDN_ERR_INVALID_ARG;
  if (scale_type != GDN_SCALE_F32 && scale_type != GDN_SCALE_E8M0) return GDN_ERR_INVALID_ARG;
  if (q8 && group && d % group) return GDN_ERR_INVALID_ARG;
  if (n_rows == 0) return GDN_OK;
  if (!x || !weight || (!y && !q8) || (q8 && !scales)) return GDN_ERR_INVALID_ARG;
  const size_t ea = dtype_size(act_dtype), er = dtype_size(res_dtype);
  if (!aligned(x, ea) || !aligned(residual, er) || !aligned(weight, 4) || !aligned(y, ea) ||
      (q8 && scale_type == GDN_SCALE_F32 && !aligned(scales, 4)))
    return GDN_ERR_INVALID_ARG;
  if (d > 32768 || n_rows > 2147483647LL) return GDN_ERR_UNSUPPORTED;
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.eps = eps;
  a.n_rows = n_rows;
  a.d = d;
  a.y = y;
  a.q8 = reinterpret_cast<uint8_t*>(q8);
  a.scales = scales;
  a.group = q8 ? group : 0;
  a.scale_type = scale_type;
  const bool vec = d % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) && aligned(y, 16) &&
                   aligned(q8, 8);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (act_dtype == GDN_BF16)
    e = res_dtype == GDN_BF16 ? dispatch_norm<__nv_bfloat16, __nv_bfloat16>(a, vec, s)
                              : dispatch_norm<__nv_bfloat16, float>(a, vec, s);
  else
    e = res_dtype == GDN_BF16 ? dispatch_norm<float, __nv_bfloat16>(a, vec, s)
                              : dispatch_norm<float, float>(a, vec, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_ADD_RMSNORM);
  return GDN_OK;
}
