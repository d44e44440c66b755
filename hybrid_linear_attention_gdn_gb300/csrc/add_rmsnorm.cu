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
// Measured: 32768 rows of 4096, bf16 with an fp32 residual, y and q8, a scale
// per row 250 us, 1.03 of the copy bandwidth (1.75 GB), per 128 values 260; with
// a bf16 residual 203 and 209 (0.88, 0.85); 64 rows 3.6 us in a graph of calls.
// With the rare exact path inlined 280 and 248 us per 128 values: its registers
// cost a CTA per SM.  4 or 6 CTAs of 256 threads instead of 5: 258 and 221, or
// 306 and 207.
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

// 8 consecutive elements as they are stored
template <typename T>
struct Vec8 {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float2 pair(int i) const {  // elements 2 i, 2 i + 1
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void put(int i, float2 x) {  // rounded to nearest even
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(x.x);
      w[2 * i + 1] = __float_as_uint(x.y);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
};
// from p[at]; VEC: p + at is 16-byte aligned and all 8 exist, else the first
// n of them (the others 0)
template <bool VEC, typename T, typename VT>
__device__ __forceinline__ void load8(Vec8<T>& f, const VT& p, int64_t at, int n) {
  if constexpr (VEC) {
    constexpr int kPer = 16 / sizeof(T);  // elements of a 16-byte access
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) {
      const uint4 u = vec_at<const uint4>(p, at + i * kPer);
      f.w[4 * i] = u.x; f.w[4 * i + 1] = u.y; f.w[4 * i + 2] = u.z; f.w[4 * i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f.put(i, make_float2(2 * i < n ? to_f32(p[at + 2 * i]) : 0.f, 2 * i + 1 < n ? to_f32(p[at + 2 * i + 1]) : 0.f));
  }
}
template <bool VEC, typename T, typename VT>
__device__ __forceinline__ void store8(const Vec8<T>& f, const VT& p, int64_t at, int n) {
  if constexpr (VEC) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i)
      vec_at<uint4>(p, at + i * kPer) = make_uint4(f.w[4 * i], f.w[4 * i + 1], f.w[4 * i + 2], f.w[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = f.pair(i);
      if (2 * i < n) p[at + 2 * i] = from_f32<T>(x.x);
      if (2 * i + 1 < n) p[at + 2 * i + 1] = from_f32<T>(x.y);
    }
  }
}

// a magnitude's bits: their order is that of the values, with NaN above all
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add2(float2 x, float2 y) { return fma2(x, both(1.f), y); }
__device__ __forceinline__ float2 sub2(float2 x, float2 y) { return fma2(y, both(-1.f), x); }
__device__ __forceinline__ uint32_t e4m3x2(float2 x) {
  return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}

// q8 is the e4m3 value nearest to y / scale before either was rounded.  The
// norm cancels from that quotient: it is 448 (h w) / max|h w|.  y times the
// scale's reciprocal is within 8 fp32 steps of it, so where 2^-20 more and
// 2^-20 less round to the same e4m3 value, that is it; else (some thirty
// values in a million) the quotient is taken exactly: from p = h w and the
// error e of that and of h, and those of the group's largest, m and me.  (The
// product alone put some ten values in a million on the wrong side.)
// 448 (p + e) / (m + me): the fp32 value nearest to it, moved off a half of an
// e4m3 step to the side of what is left, so that rounding to e4m3 is the only
// rounding.  What is left is 448 p - z m and the errors' part.  On a half z has
// five significant bits: the product's two pieces and z m cancel exactly, so
// that where h w lost nothing (e = me = 0, as with 16-bit h and w) a quotient
// that is the half stays on it.  (The remainder of the division instead, z and
// t both rounded, moved those off to either side.)
__device__ __forceinline__ float quotient(float p, float e, float m, float me, float im) {
  const float t = p * im, r = fmaf(-t, m, p) + fmaf(-t, me, e);
  const float z = fmaf(448.f, t, r * im * 448.f), a = __fmul_rn(448.f, p);
  const float rest = (fmaf(-z, m, a) + fmaf(448.f, p, -a)) + fmaf(448.f, e, -__fmul_rn(z, me));
  const uint32_t u = __float_as_uint(z);
  if (rest == 0.f) return z;
  return __uint_as_float((u - ((u ^ __float_as_uint(rest)) >> 31)) | 1u);
}

__device__ __forceinline__ float2 unpack(uint32_t bf16x2) {
  return make_float2(__uint_as_float(bf16x2 << 16), __uint_as_float(bf16x2 & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float2 x) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// Four pairs of a vector: the sums h, what their rounding lost, the weights.
struct Four {
  float2 h[4];
  uint32_t lost[4];
  float2 g[4];
  float i2;
  __device__ __forceinline__ float2 product(int i) const { return mul2(mul2(h[i], both(i2)), g[i]); }  // h w
  // what the roundings of the sum and of the product p left
  __device__ __forceinline__ float2 error(int i, float2 p) const {
    return fma2(mul2(unpack(lost[i]), both(i2)), g[i], fma2(mul2(h[i], both(i2)), g[i], mul2(p, both(-1.f))));
  }
  // the error of the largest, |h w| = m: of several the largest in its direction
  __device__ __forceinline__ float error_of(uint32_t m, float me) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = product(i);
      if (mag(p.x) != m && mag(p.y) != m) continue;
      const float2 e = error(i, p);
      if (mag(p.x) == m) me = fmaxf(me, p.x < 0.f ? -e.x : e.x);
      if (mag(p.y) == m) me = fmaxf(me, p.y < 0.f ? -e.y : e.y);
    }
    return me;
  }
};
constexpr float kNone = -3.4e38f;  // no error yet

// The exact values of a vector, by all lanes of a warp; gl: lanes of a group,
// which find me together.  Not inlined: it is rare, and what it needs would
// take registers (and with them CTAs) from every row.
__device__ __noinline__ uint2 exact_q8(const Four f, uint32_t mu, int gl) {
  float me = f.error_of(mu, kNone);
  for (int o = 1; o < gl; o <<= 1) me = fmaxf(me, __shfl_xor_sync(0xffffffffu, me, o));
  const float m = __uint_as_float(mu), im = 1.f / m;
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = f.product(i), e = f.error(i, p);
    q[i >> 1] |= e4m3x2(make_float2(quotient(p.x, e.x, m, me, im), quotient(p.y, e.y, m, me, im))) << (16 * (i & 1));
  }
  return make_uint2(q[0], q[1]);
}

// the same where p = h w and its errors are at hand, and me known
struct FourP {
  float2 p[4];
  uint32_t e[4];
};
__device__ __noinline__ uint2 exact_q8_of(const FourP f, float m, float me) {
  const float im = 1.f / m;
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = f.p[i], e = unpack(f.e[i]);
    q[i >> 1] |= e4m3x2(make_float2(quotient(p.x, e.x, m, me, im), quotient(p.y, e.y, m, me, im))) << (16 * (i & 1));
  }
  return make_uint2(q[0], q[1]);
}

// the scale of a group whose largest |y| is top, stored at index `at`; returns
// 1 / scale (0 only for an infinite scale).  e4m3's largest value is 448.
__device__ __forceinline__ float put_scale(const NormArgs& a, float top, int64_t at, int64_t n_scales, bool store) {
  if (a.scale_type == GDN_SCALE_F32) {
    // at least 2^-126: a smaller scale's reciprocal could overflow
    float s = top == 0.f ? 1.f : top * (1.f / 448.f);
    s = s < 1.17549435e-38f ? 1.17549435e-38f : s;
    if (store) GDN_GV(reinterpret_cast<float*>(a.scales), n_scales)[at] = s;
    return __fdividef(1.f, s);
  }
  // byte b stands for 2^(b - 127): the smallest with 448 * 2^(b - 127) >= top
  int b = 127;
  if (top != top) {
    b = 255;
  } else if (top > 0.f) {
    const float s = top / 448.f;
    const uint32_t u = __float_as_uint(s);
    // the exponent, rounded up; byte 0 is the subnormal 2^-127
    b = u > 0x400000u ? (int)(u >> 23) + ((u & 0x7fffffu) ? 1 : 0) : 0;
    // the division may have rounded down onto a power of two below top / 448
    if (b < 254 && b > 0 && 448.f * __uint_as_float((uint32_t)b << 23) < top) ++b;
    b = b > 254 ? 254 : b;
  }
  if (store) GDN_GV(reinterpret_cast<uint8_t*>(a.scales), n_scales)[at] = (uint8_t)b;
  if (b == 255) return __uint_as_float(0x7fc00000u);
  // 2^(127 - b) as a float: normal for b <= 253, subnormal for 254
  return b < 254 ? __uint_as_float((uint32_t)(254 - b) << 23) : 5.87747175e-39f;
}

// TPR threads per row, ROWS rows per CTA
template <typename Tact, typename Tres, int TPR, int ROWS, int V, bool VEC, bool ROWSCALE>
__global__ void __launch_bounds__(TPR* ROWS, TPR* ROWS >= 1024 ? 1 : 1280 / (TPR * ROWS))
    add_rmsnorm_kernel(const NormArgs a) {
  constexpr int kRowWarps = TPR / 32;
  __shared__ uint64_t red[ROWS][32];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x % TPR, rloc = threadIdx.x / TPR, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * ROWS + rloc;
  const bool live = row < a.n_rows;  // the same for the threads of a row
  const int64_t n = a.n_rows * a.d, base = row * a.d;
  const auto x = GDN_GV(reinterpret_cast<const Tact*>(a.x), n);
  const auto res = GDN_GV(reinterpret_cast<Tres*>(a.residual), n);
  const auto w = GDN_GV(a.weight, a.d);
  float2 h[V][4];      // x + residual
  uint32_t lost[V][4];  // what its rounding lost, as bf16 pairs
  {
    Vec8<Tact> xv[V];
    Vec8<Tres> rv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * TPR + t);
#pragma unroll
      for (auto& u : xv[v].w) u = 0u;
#pragma unroll
      for (auto& u : rv[v].w) u = 0u;
      if (live && c < a.d) {
        load8<VEC>(xv[v], x, base + c, a.d - c);
        if (a.residual) load8<VEC>(rv[v], res, base + c, a.d - c);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * TPR + t);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 xi = xv[v].pair(i), ri = rv[v].pair(i), s = add2(xi, ri), b = sub2(s, xi);
        h[v][i] = s;
        lost[v][i] = pack(add2(sub2(xi, sub2(s, b)), sub2(ri, b)));
        rv[v].put(i, s);
      }
      if (a.residual && live && c < a.d) store8<VEC>(rv[v], res, base + c, a.d - c);
    }
  }
  float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) ss2 = fma2(h[v][i], h[v][i], ss2);
  // over the row's threads
  auto row_all = [&](auto m, auto join) {
#pragma unroll
    for (int o = 16; o; o >>= 1) m = join(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (kRowWarps > 1) {
      auto* const part = reinterpret_cast<decltype(m)*>(red[rloc]);
      __syncthreads();  // red has been read
      if (lane == 0) part[t >> 5] = m;
      __syncthreads();
      m = part[lane % kRowWarps];
#pragma unroll
      for (int o = kRowWarps / 2; o; o >>= 1) m = join(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    return m;
  };
  const float ss = row_all(ss2.x + ss2.y, [](float p, float q) { return p + q; });
  const float inv = 1.f / sqrtf(ss / (float)a.d + a.eps);
  // inv = i2 c2 with a power of two i2, so that h i2 w neither overflows nor
  // vanishes before it is scaled
  const uint32_t ib = __float_as_uint(inv);
  const bool normal = inv > 1.17549435e-38f && inv < 3.4e38f;
  const float i2 = normal ? __uint_as_float(ib & 0x7f800000u) : inv;
  const float c2 = normal ? __uint_as_float((ib & 0x7fffffu) | 0x3f800000u) : 1.f;
  auto four = [&](int v, const Vec8<float>& g) {
    Four f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.h[i] = h[v][i];
      f.lost[i] = lost[v][i];
      f.g[i] = g.pair(i);
    }
    f.i2 = i2;
    return f;
  };
  const int64_t per_row = ROWSCALE ? 1 : a.group ? a.d / a.group : 1, n_scales = a.n_rows * per_row;
  // One scale per row: p = h w in place of h and its error in place of what h
  // lost, y, and the row's largest |p| with its error (of several as large,
  // the largest in its direction): one maximum of both.
  float row_m = 0.f, row_me = 0.f, row_inv = 0.f;
  if constexpr (ROWSCALE) {
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * TPR + t);
      if (live && c < a.d) {
        Vec8<float> g;
        Vec8<Tact> y;
        load8<VEC>(g, w, c, a.d - c);
        const Four f = four(v, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = f.product(i);
          lost[v][i] = pack(f.error(i, p));
          h[v][i] = p;
          y.put(i, mul2(p, both(c2)));
          top = max(top, max(mag(p.x), mag(p.y)));
        }
        if (a.y) store8<VEC>(y, GDN_GV(reinterpret_cast<Tact*>(a.y), n), base + c, a.d - c);
      }
    }
    float me = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = h[v][i], e = unpack(lost[v][i]);
        if (mag(p.x) == top) me = fmaxf(me, p.x < 0.f ? -e.x : e.x);
        if (mag(p.y) == top) me = fmaxf(me, p.y < 0.f ? -e.y : e.y);
      }
    const uint32_t eb = __float_as_uint(me), order = eb ^ (eb >> 31 ? 0xffffffffu : 0x80000000u);
    const uint64_t key = row_all((uint64_t)top << 32 | order, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
    const uint32_t ob = (uint32_t)key;
    row_m = __uint_as_float((uint32_t)(key >> 32));
    row_me = __uint_as_float(ob ^ (ob >> 31 ? 0x80000000u : 0xffffffffu));
    if (live) row_inv = put_scale(a, row_m * c2, row, n_scales, t == 0);
  }
  const auto q8 = GDN_GV(a.q8, n);
  const int gl = a.group / 8;  // lanes of a group
  auto put_q8 = [&](int c, uint2 q) {
    if constexpr (VEC) {
      vec_at<uint2>(q8, base + c) = q;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < a.d - c) q8[base + c + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
  };
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * TPR + t);
    const bool in = live && c < a.d;
    Vec8<float> g = {};
    float2 p[4];
    float m = row_m, inv_s = row_inv;
    if constexpr (ROWSCALE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = h[v][i];
    } else {
      if (in) load8<VEC>(g, w, c, a.d - c);
      const Four f = four(v, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = f.product(i);
      if (a.y && in) {
        Vec8<Tact> y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.put(i, mul2(p[i], both(c2)));
        store8<VEC>(y, GDN_GV(reinterpret_cast<Tact*>(a.y), n), base + c, a.d - c);
      }
      if (!a.q8) continue;
      uint32_t mu = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) mu = max(mu, max(mag(p[i].x), mag(p[i].y)));
      for (int o = 1; o < gl; o <<= 1) mu = max(mu, __shfl_xor_sync(0xffffffffu, mu, o));
      m = __uint_as_float(mu);
      if (in) inv_s = put_scale(a, m * c2, row * per_row + c / a.group, n_scales, t % gl == 0);
    }
    const float k = c2 * inv_s;
    // (within these the quotient's pieces neither overflow nor vanish)
    const bool exact = in && a.scale_type == GDN_SCALE_F32 && m > 1e-24f && m < 1e24f;
    const float2 lo = both(exact ? k * (1.f - 0x1p-20f) : k), hi = both(exact ? k * (1.f + 0x1p-20f) : k);
    uint32_t q[2] = {0u, 0u}, differ = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = e4m3x2(mul2(p[i], lo));
      q[i >> 1] |= b << (16 * (i & 1));
      differ |= b ^ e4m3x2(mul2(p[i], hi));
    }
    if (__any_sync(0xffffffffu, differ)) {
      uint2 z;
      if constexpr (ROWSCALE) {
        FourP f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f.p[i] = p[i];
          f.e[i] = lost[v][i];
        }
        z = exact_q8_of(f, m, row_me);
      } else {
        z = exact_q8(four(v, g), __float_as_uint(m), gl);
      }
      if (differ) {
        q[0] = z.x;
        q[1] = z.y;
      }
    }
    if (in) put_q8(c, make_uint2(q[0], q[1]));
  }
}

template <typename Tact, typename Tres, int TPR, int ROWS, int V>
cudaError_t launch_norm(const NormArgs& a, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)((a.n_rows + ROWS - 1) / ROWS)), block(TPR * ROWS);
  if (a.q8 && a.group == 0)
    return vec ? launch_pdl(add_rmsnorm_kernel<Tact, Tres, TPR, ROWS, V, true, true>, grid, block, 0, s, dim3(1), a)
               : launch_pdl(add_rmsnorm_kernel<Tact, Tres, TPR, ROWS, V, false, true>, grid, block, 0, s, dim3(1), a);
  return vec ? launch_pdl(add_rmsnorm_kernel<Tact, Tres, TPR, ROWS, V, true, false>, grid, block, 0, s, dim3(1), a)
             : launch_pdl(add_rmsnorm_kernel<Tact, Tres, TPR, ROWS, V, false, false>, grid, block, 0, s, dim3(1), a);
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
