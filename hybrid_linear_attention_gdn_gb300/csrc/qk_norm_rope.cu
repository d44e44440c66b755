// Norms of queries and keys per head, rotation by position, and the write of
// keys and values to their cache pages, in one pass.  Not written on the
// pages; the published blocks: RMS norm of each head (Henry et al., "Query-Key
// Normalization", 2020) and rotary embedding (Su et al., "RoFormer", 2021).
//   y = x / sqrt(mean(x^2) + eps) * w
//   pairs (a, b) of y's first rot values -> (a c - b s, b c + a s)
// The row's position picks c and s from a table that the caller computed (in
// double: an fp32 angle of a far position is off by its own size).  The slot
// map of gdn_batch_maps says where a row's k and v go.
//
// HBM bound: each value is read and written once.
//
// qk_rope_kernel (head sizes 8 to 256, powers of two): a warp walks heads of one
// row, whose cosines and sines it holds in registers, four heads' (or
// groups of small heads') loads in flight.  A lane has 8 values of a head, in two runs of
// 4 that are each other's partners, so that nothing but the sum of squares goes
// between lanes.  qk_rope_any_kernel: every other shape, a warp per head.
#include "gdn_common.cuh"
#include "decode_tma.cuh"  // sm_count

namespace gdn {
namespace {

struct RopeArgs {
  int32_t hq, hk, hv, d, dv, rot, interleaved;
  int64_t n_rows;
  gdn_rows q, k, v, q_out, k_out;
  gdn_pages k_cache, v_cache;
  const float* q_weight;
  const float* k_weight;
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  const int64_t* positions;
  const int64_t* slot_map;
  int64_t n_slots;  // num_pages << shift
  int32_t shift;
  int32_t k_to_out, to_cache;
  uint32_t* err;
};

constexpr int kThreads = 256;

// The extent of rows x heads x width elements at these strides.
__device__ __forceinline__ long long extent(int64_t rows, int64_t row, int heads, int64_t head, int width) {
  return rows > 0 && heads > 0 ? (rows - 1) * row + (heads - 1) * head + width : 0;
}

// What a row's position and slot say.  cls: 0 live, 1 position outside the
// table (outputs are zeros); slot -1: nothing goes to the cache.
struct RowInfo {
  int64_t pos, slot;
  bool bad;
};
__device__ __forceinline__ RowInfo row_info(const RopeArgs& a, int64_t r, bool leader) {
  RowInfo i;
  i.pos = GDN_GV(a.positions, a.n_rows)[r];
  i.bad = i.pos < 0 || i.pos >= a.max_pos;
  if (i.bad && leader) report(a.err, GDN_DEV_ERR_SEQLENS);
  i.slot = -1;
  if (a.to_cache) {
    const int64_t s = GDN_GV(a.slot_map, a.n_rows)[r];
    if (s >= 0 && s < a.n_slots) i.slot = i.bad ? -1 : s;
    else if (s != -1 && leader) report(a.err, GDN_DEV_ERR_SLOT_OOB);
  }
  if (i.bad) i.pos = 0;
  return i;
}
__device__ __forceinline__ int64_t page_off(const RopeArgs& a, const gdn_pages& c, int64_t slot, int h) {
  return (slot >> a.shift) * c.page + (slot & (((int64_t)1 << a.shift) - 1)) * c.row + h * c.head;
}
__device__ __forceinline__ long long page_extent(const RopeArgs& a, const gdn_pages& c, int heads, int width) {
  const int64_t b = (int64_t)1 << a.shift;
  return a.n_slots > 0 && heads > 0 ? ((a.n_slots >> a.shift) - 1) * c.page + (b - 1) * c.row + (heads - 1) * c.head + width
                                    : 0;
}

// Every shape: a warp per head, the head's normed values in shared memory.
template <typename T>
__global__ void __launch_bounds__(kThreads) qk_rope_any_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) float smem[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto y = GDN_SV(smem + warp * a.d, a.d);
  const int heads = a.hq + a.hk + (a.to_cache ? a.hv : 0);
  const int64_t items = a.n_rows * heads;
  const int half = a.rot / 2;
  const auto tab = GDN_GV(a.cos_sin, a.max_pos * a.rot);
  for (int64_t it = (int64_t)blockIdx.x * (kThreads / 32) + warp; it < items; it += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t r = it / heads;
    const int hh = (int)(it % heads);
    const RowInfo ri = row_info(a, r, hh == 0 && lane == 0);
    if (hh >= a.hq + a.hk) {  // a value head to its page
      const int h = hh - a.hq - a.hk;
      if (ri.slot < 0) continue;
      const auto src = GDN_GV((const T*)a.v.data, extent(a.n_rows, a.v.row, a.hv, a.v.head, a.dv)) + (r * a.v.row + h * a.v.head);
      const auto dst = GDN_GV((T*)a.v_cache.data, page_extent(a, a.v_cache, a.hv, a.dv)) + page_off(a, a.v_cache, ri.slot, h);
      for (int e = lane; e < a.dv; e += 32) dst[e] = src[e];
      continue;
    }
    const bool isq = hh < a.hq;
    const int h = isq ? hh : hh - a.hq;
    const gdn_rows& in = isq ? a.q : a.k;
    const int nh = isq ? a.hq : a.hk;
    const auto src = GDN_GV((const T*)in.data, extent(a.n_rows, in.row, nh, in.head, a.d)) + (r * in.row + h * in.head);
    float ss = 0.f;
    for (int e = lane; e < a.d; e += 32) {
      const float x = to_f32(src[e]);
      y[e] = x;
      ss = fmaf(x, x, ss);
    }
#pragma unroll
    for (int o = 16; o; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float* const wp = isq ? a.q_weight : a.k_weight;
    const float rn = wp ? 1.f / sqrtf(ss / a.d + a.eps) : 1.f;
    const auto w = GDN_GV(wp, a.d);
    __syncwarp();
    auto normed = [&](int e) { return wp ? y[e] * rn * w[e] : y[e]; };
    auto value = [&](int e) {
      if (ri.bad) return 0.f;
      if (e >= a.rot) return normed(e);
      const int i = a.interleaved ? e >> 1 : e < half ? e : e - half;  // the pair
      const bool first = a.interleaved ? !(e & 1) : e < half;
      const int other = a.interleaved ? e ^ 1 : first ? e + half : e - half;
      const float c = tab[ri.pos * a.rot + i], s = tab[ri.pos * a.rot + half + i];
      const float u = normed(e), t = normed(other);
      return first ? u * c - t * s : u * c + t * s;
    };
    // every value is read (from shared memory) before any output is written
    for (int e = lane; e < a.d; e += 32) {
      const T o = from_f32<T>(value(e));
      if (isq) {
        (GDN_GV((T*)a.q_out.data, extent(a.n_rows, a.q_out.row, a.hq, a.q_out.head, a.d)) +
         (r * a.q_out.row + h * a.q_out.head))[e] = o;
      } else {
        if (a.k_to_out)
          (GDN_GV((T*)a.k_out.data, extent(a.n_rows, a.k_out.row, a.hk, a.k_out.head, a.d)) +
           (r * a.k_out.row + h * a.k_out.head))[e] = o;
        if (ri.slot >= 0)
          (GDN_GV((T*)a.k_cache.data, page_extent(a, a.k_cache, a.hk, a.d)) + page_off(a, a.k_cache, ri.slot, h))[e] = o;
      }
    }
    __syncwarp();
  }
}

// 4 consecutive values
template <typename T> struct Four;
template <> struct Four<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void get(float* f) const {
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    u.x = *reinterpret_cast<const uint32_t*>(&a);
    u.y = *reinterpret_cast<const uint32_t*>(&b);
  }
};
template <> struct Four<float> {
  float4 u;
  __device__ __forceinline__ void get(float* f) const { f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w; }
  __device__ __forceinline__ void set(const float* f) { u = make_float4(f[0], f[1], f[2], f[3]); }
};

// grid x: rows x parts of their heads, a warp each.  LPH = d / 8 lanes per head.
constexpr int kAhead = 4;  // head groups whose loads are in flight
template <typename T, int LPH, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) qk_rope_kernel(const RopeArgs a, const int parts) {
  using F = Four<T>;
  constexpr int HPW = 32 / LPH, D = 8 * LPH;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, l = lane % LPH, hsub = lane / LPH;
  const int64_t wi = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t r = wi / parts;
  const int part = (int)(wi % parts);
  if (r >= a.n_rows) return;
  const RowInfo ri = row_info(a, r, part == 0 && lane == 0);
  // the lane's two runs of 4 values
  const int half = a.rot / 2;
  const bool turns = 8 * l < a.rot;  // (rot is a multiple of 8)
  const int ea = INTER || !turns ? 8 * l : 4 * l, eb = INTER || !turns ? 8 * l + 4 : half + 4 * l;
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns && !ri.bad) {  // (a table of no rows is not read)
    const auto tab = GDN_GV(a.cos_sin, a.max_pos * a.rot) + ri.pos * a.rot;
    const float4 c4 = vec_at<const float4>(tab, 4 * l), s4 = vec_at<const float4>(tab, half + 4 * l);
    c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
    s[0] = s4.x, s[1] = s4.y, s[2] = s4.z, s[3] = s4.w;
  }
  // Head groups i0, i0 + parts, .. of nh heads from src to out and cache (which
  // may be null), all at the row; strides of heads in 32 bits.
  auto walk = [&](const auto src, const auto out, const auto cache, const bool to_out, const bool to_cache, const int nh,
                  const int in_head, const int out_head, const int c_head, const float* const wp, const int i0) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (wp) {
      const auto wv = GDN_GV(wp, D);
      const float4 wa = vec_at<const float4>(wv, ea), wb = vec_at<const float4>(wv, eb);
      w[0] = wa.x, w[1] = wa.y, w[2] = wa.z, w[3] = wa.w, w[4] = wb.x, w[5] = wb.y, w[6] = wb.z, w[7] = wb.w;
    }
    const int step = HPW * parts;
    for (int h0 = i0 * HPW + hsub; h0 - hsub < nh; h0 += kAhead * step) {
      F xa[kAhead], xb[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (h0 + k * step < nh) {
          xa[k] = vec_at<const F>(src, (h0 + k * step) * in_head + ea);
          xb[k] = vec_at<const F>(src, (h0 + k * step) * in_head + eb);
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int h = h0 + k * step;
        if (h - hsub >= nh) break;  // the whole warp
        float y[8];
        xa[k].get(y);  // (a head beyond the last one: whatever, and not stored)
        xb[k].get(y + 4);
        if (wp) {
          float2 sq = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 v = make_float2(y[e], y[e + 1]);
            sq = fma2(v, v, sq);
          }
          float ss = sq.x + sq.y;
#pragma unroll
          for (int o = LPH / 2; o; o /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float rn = rsqrtf(ss * (1.f / D) + a.eps);  // 2 units in the last place
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 v = mul2(make_float2(y[e], y[e + 1]), mul2(make_float2(w[e], w[e + 1]), make_float2(rn, rn)));
            y[e] = v.x;
            y[e + 1] = v.y;
          }
        }
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& u = y[INTER ? 2 * e : e];
            float& t = y[INTER ? 2 * e + 1 : e + 4];
            const float p = u * c[e] - t * s[e];
            t = t * c[e] + u * s[e];
            u = p;
          }
        }
        if (ri.bad)
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = 0.f;
        F oa, ob;
        oa.set(y);
        ob.set(y + 4);
        if (to_out && h < nh) {
          vec_at<F>(out, h * out_head + ea) = oa;
          vec_at<F>(out, h * out_head + eb) = ob;
        }
        if (to_cache && h < nh) {
          vec_at<F>(cache, h * c_head + ea) = oa;
          vec_at<F>(cache, h * c_head + eb) = ob;
        }
      }
    }
  };
  // queries first, then keys: group i of both in turn to part i % parts
  const int nq = (a.hq + HPW - 1) / HPW;
  {
    const auto src = GDN_GV((const T*)a.q.data, extent(a.n_rows, a.q.row, a.hq, a.q.head, D)) + (a.hq ? r * a.q.row : 0);
    const auto out = GDN_GV((T*)a.q_out.data, extent(a.n_rows, a.q_out.row, a.hq, a.q_out.head, D)) +
                     (a.hq ? r * a.q_out.row : 0);
    walk(src, out, out, true, false, a.hq, (int)a.q.head, (int)a.q_out.head, 0, a.q_weight, part);
  }
  {
    const bool to_out = a.k_to_out, to_cache = ri.slot >= 0;
    const auto src = GDN_GV((const T*)a.k.data, extent(a.n_rows, a.k.row, a.hk, a.k.head, D)) + (a.hk ? r * a.k.row : 0);
    const auto out = GDN_GV((T*)a.k_out.data, to_out ? extent(a.n_rows, a.k_out.row, a.hk, a.k_out.head, D) : 0) +
                     (to_out && a.hk ? r * a.k_out.row : 0);
    const auto cache = GDN_GV((T*)a.k_cache.data, to_cache ? page_extent(a, a.k_cache, a.hk, D) : 0) +
                       (to_cache ? page_off(a, a.k_cache, ri.slot, 0) : 0);
    walk(src, out, cache, to_out, to_cache, a.hk, (int)a.k.head, (int)a.k_out.head, (int)a.k_cache.head, a.k_weight,
         ((part - nq) % parts + parts) % parts);
  }
  if (a.to_cache && ri.slot >= 0 && a.hv > 0) {  // values: 4 at a time
    const int n4 = a.dv / 4, n = a.hv * n4;
    const auto src = GDN_GV((const T*)a.v.data, extent(a.n_rows, a.v.row, a.hv, a.v.head, a.dv)) + r * a.v.row;
    const auto dst = GDN_GV((T*)a.v_cache.data, page_extent(a, a.v_cache, a.hv, a.dv));
    for (int e0 = part * 32 + lane; e0 < n; e0 += kAhead * parts * 32) {
      F x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int e = e0 + k * parts * 32;
        if (e < n) x[k] = vec_at<const F>(src, e / n4 * a.v.head + e % n4 * 4);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int e = e0 + k * parts * 32;
        if (e < n) vec_at<F>(dst, page_off(a, a.v_cache, ri.slot, e / n4) + e % n4 * 4) = x[k];
      }
    }
  }
}

// whether the vectorised kernel takes these tensors: 4 values are one access everywhere
// and a head's place in its row is a 32-bit offset
bool small(int64_t head, int heads) { return head * heads < (1LL << 30); }
bool vec_rows(const gdn_rows& r, int heads, size_t esz) {
  return heads == 0 || !r.data || (aligned(r.data, 4 * esz) && r.row % 4 == 0 && r.head % 4 == 0 && small(r.head, heads));
}
bool vec_pages(const gdn_pages& r, int heads, size_t esz) {
  return heads == 0 || !r.data ||
         (aligned(r.data, 4 * esz) && r.page % 4 == 0 && r.row % 4 == 0 && r.head % 4 == 0 && small(r.head, heads));
}
bool vec_shape(const RopeArgs& a, size_t esz) {
  if (a.d < 8 || a.d > 256 || (a.d & (a.d - 1)) || a.rot % 8 || !aligned(a.cos_sin, 16) || !aligned(a.q_weight, 16) ||
      !aligned(a.k_weight, 16))
    return false;
  if (!vec_rows(a.q, a.hq, esz) || !vec_rows(a.q_out, a.hq, esz) || !vec_rows(a.k, a.hk, esz) ||
      !vec_rows(a.k_out, a.hk, esz))
    return false;
  return !a.to_cache || (vec_pages(a.k_cache, a.hk, esz) &&
                         (a.hv == 0 || (a.dv % 4 == 0 && vec_rows(a.v, a.hv, esz) && vec_pages(a.v_cache, a.hv, esz))));
}

template <typename T, int LPH>
cudaError_t rope_vec(const RopeArgs& a, cudaStream_t s) {
  constexpr int HPW = 32 / LPH;
  // A row's heads in so many parts that there are 8 warps per SM: a warp's
  // start (position, table, weights) costs as much as several heads, so that
  // more than one part per row is for few rows only (32768 rows of 32 + 4 heads
  // 117 us in one part, 148 in two; 64 rows 3 us in 18 parts, 4 in 5).
  const int64_t groups = (a.hq + HPW - 1) / HPW + (a.hk + HPW - 1) / HPW;
  const int64_t want = (8LL * sm_count() + a.n_rows - 1) / a.n_rows;
  const int parts = (int)std::max<int64_t>(1, std::min(want, groups));
  const int64_t ctas = (a.n_rows * parts + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 2147483647LL) return cudaErrorInvalidValue;
  return a.interleaved ? launch_pdl(qk_rope_kernel<T, LPH, true>, dim3((unsigned)ctas), dim3(kThreads), 0, s, dim3(1), a, parts)
                       : launch_pdl(qk_rope_kernel<T, LPH, false>, dim3((unsigned)ctas), dim3(kThreads), 0, s, dim3(1), a, parts);
}
template <typename T>
cudaError_t rope_any(const RopeArgs& a, cudaStream_t s);
template <typename T>
cudaError_t rope_dispatch(const RopeArgs& a, cudaStream_t s) {
  if (vec_shape(a, sizeof(T))) switch (a.d) {
      case 8: return rope_vec<T, 1>(a, s);
      case 16: return rope_vec<T, 2>(a, s);
      case 32: return rope_vec<T, 4>(a, s);
      case 64: return rope_vec<T, 8>(a, s);
      case 128: return rope_vec<T, 16>(a, s);
      case 256: return rope_vec<T, 32>(a, s);
    }
  return rope_any<T>(a, s);
}

template <typename T>
cudaError_t rope_any(const RopeArgs& a, cudaStream_t s) {
  const int64_t items = a.n_rows * (a.hq + a.hk + (a.to_cache ? a.hv : 0));
  const int64_t want = (items + kThreads / 32 - 1) / (kThreads / 32), most = 8LL * sm_count();
  return launch_pdl(qk_rope_any_kernel<T>, dim3((unsigned)std::min(want, most)), dim3(kThreads),
                    sizeof(float) * (kThreads / 32) * a.d, s, dim3(1), a);
}

bool bad_rows(const gdn_rows& r, size_t esz) { return !r.data || r.row < 0 || r.head < 0 || !aligned(r.data, esz); }
bool bad_pages(const gdn_pages& r, size_t esz) {
  return !r.data || r.page < 0 || r.row < 0 || r.head < 0 || !aligned(r.data, esz);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_qk_norm_rope(int32_t act_dtype, int32_t hq, int32_t hk, int32_t d, int32_t hv, int32_t dv,
                                       int64_t n_rows, gdn_rows q, gdn_rows k, gdn_rows v, const float* q_weight,
                                       const float* k_weight, float eps, const float* cos_sin, int64_t max_pos,
                                       int32_t rot, int32_t interleaved, const int64_t* positions, gdn_rows q_out,
                                       gdn_rows k_out, gdn_pages k_cache, gdn_pages v_cache, int32_t num_pages,
                                       int32_t block, const int64_t* slot_map, uint32_t* dev_err, void* stream) {
  using namespace gdn;
  if (act_dtype != GDN_F32 && act_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  const size_t esz = dtype_size(act_dtype);
  if (hq < 0 || hk < 0 || hq + (int64_t)hk <= 0 || hv < 0 || d <= 0 || n_rows < 0 || num_pages < 0)
    return GDN_ERR_INVALID_ARG;
  if (rot < 0 || rot > d || rot % 2 || max_pos < 0 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const bool cache = slot_map != nullptr;
  if (cache && (hk <= 0 || block <= 0 || (block & (block - 1)) || (hv > 0 && dv <= 0))) return GDN_ERR_INVALID_ARG;
  if (d > 1024 || dv > 1024 || hq > 65535 || hk > 65535 || hv > 65535 || interleaved < 0 || interleaved > 1)
    return GDN_ERR_UNSUPPORTED;
  if (n_rows == 0) return GDN_OK;
  if (n_rows > 2147483647LL) return GDN_ERR_UNSUPPORTED;
  if (!positions || (rot > 0 && max_pos > 0 && !cos_sin) || !aligned(cos_sin, 4)) return GDN_ERR_INVALID_ARG;
  if (hq > 0 && (bad_rows(q, esz) || bad_rows(q_out, esz))) return GDN_ERR_INVALID_ARG;
  if (hk > 0 && bad_rows(k, esz)) return GDN_ERR_INVALID_ARG;
  if (hk > 0 && !cache && bad_rows(k_out, esz)) return GDN_ERR_INVALID_ARG;
  if (k_out.data && bad_rows(k_out, esz)) return GDN_ERR_INVALID_ARG;
  if (cache && num_pages > 0 && (bad_pages(k_cache, esz) || (hv > 0 && (bad_rows(v, esz) || bad_pages(v_cache, esz)))))
    return GDN_ERR_INVALID_ARG;
  RopeArgs a = {};
  a.hq = hq;
  a.hk = hk;
  a.hv = hv;
  a.d = d;
  a.dv = dv;
  a.rot = rot;
  a.interleaved = interleaved;
  a.n_rows = n_rows;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_out = k_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.cos_sin = cos_sin;
  a.max_pos = max_pos;
  a.positions = positions;
  a.slot_map = slot_map;
  a.to_cache = cache;
  a.k_to_out = k_out.data != nullptr;
  if (cache) {
    while ((1 << a.shift) < block) ++a.shift;
    a.n_slots = (int64_t)num_pages << a.shift;
  }
  a.err = dev_err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = act_dtype == GDN_BF16 ? rope_dispatch<__nv_bfloat16>(a, s) : rope_dispatch<float>(a, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_QK_NORM_ROPE);
  return GDN_OK;
}
