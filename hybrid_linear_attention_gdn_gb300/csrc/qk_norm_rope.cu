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
#include "ssm.cuh"  // allow_smem
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
  if (!positions || (rot > 0 && !cos_sin) || !aligned(cos_sin, 4)) return GDN_ERR_INVALID_ARG;
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
  const cudaError_t e = act_dtype == GDN_BF16 ? rope_any<__nv_bfloat16>(a, s) : rope_any<float>(a, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_QK_NORM_ROPE);
  return GDN_OK;
}
