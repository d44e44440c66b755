// Linear attention with a fixed decay per head: entry points, the decode step
// and the prefill's token recurrence.  Not written on the pages; the published
// step (Sun et al., "Retentive Network", 2023; Qin et al., "Lightning
// Attention-2", 2024) over the slot pools of the other layers:
//   S <- lambda S + k v^T,  o = scale S^T q,  lambda = exp(log_decay)
#include "lin.cuh"

#include "decode_tma.cuh"  // sm_count

#include <cstring>

namespace gdn {
namespace {

using namespace lin;

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
// A state row of dk floats lies across LPR = dk / 4 lanes, a float4 each; a
// thread holds NR of its warp's rows at once, all requested before the first
// is used.  HBM bound: 8 dk bytes per row against 4 dk flops; 249 requests of 32
// heads of 128 x 128 153 us, a copy's rate, one request 2.0 us.  NR 4 of dk 128, 32
// rows per CTA: with 8 as fast from 64 requests on, but 2.5 us for one and 9.3
// for 16 of them (7.8); with 16 192 us for 249, as half the warps fit.
struct DecodeArgs {
  float* ssm;
  int32_t num_slots;
  const float* log_decay;
  float scale;
  const int32_t* slot_ids;
  const void* qkv;
  void* out;
  uint32_t* err;
  int32_t B, hk, hv, dv, G;
  int64_t C;
  int32_t vec;  // q and k in 4-element accesses
};

constexpr int kDT = 256;

template <int DK, int NR, typename T>
__global__ void __launch_bounds__(kDT) lin_decode_kernel(const DecodeArgs a) {
  constexpr int LPR = DK / 4, RPW = 32 / LPR, ROWS = kDT / 32 * RPW * NR;
  static_assert(NR <= LPR, "the reduction gives each lane at most one row");
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z;
  const int32_t slot = GDN_GV(a.slot_ids, a.B)[b];
  const auto x = GDN_GV(reinterpret_cast<const T*>(a.qkv), a.B * a.C) + b * a.C;
  const int row0 = blockIdx.x * ROWS + warp * RPW * NR + lane / LPR;  // rows row0 + i RPW
  const int col = lane % LPR * 4;
  const int64_t kd = (int64_t)a.hk * DK, hq = h / a.G;
  float4 q, k;
  auto load4 = [&](int64_t at) {
    if (a.vec) {
      if constexpr (sizeof(T) == 2) {
        const uint2 u = vec_at<const uint2>(x, at);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
      } else {
        return vec_at<const float4>(x, at);
      }
    }
    return make_float4(to_f32(x[at]), to_f32(x[at + 1]), to_f32(x[at + 2]), to_f32(x[at + 3]));
  };
  q = load4(hq * DK + col);
  k = load4(kd + hq * DK + col);
  float v[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) v[i] = row0 + i * RPW < a.dv ? to_f32(x[2 * kd + (int64_t)h * a.dv + row0 + i * RPW]) : 0.f;
  const Decay dec = decay_of(GDN_GV(a.log_decay, a.hv)[h]);
  const int cls = slot_class(slot, a.num_slots);
  const auto out = GDN_GV(reinterpret_cast<T*>(a.out), (long long)a.B * a.hv * a.dv) + ((int64_t)b * a.hv + h) * a.dv;
  float p[NR];
  if (cls == 0) {
    const int64_t head = (int64_t)a.dv * DK;
    const auto S = GDN_GV(a.ssm, a.num_slots * a.hv * head) + ((int64_t)slot * a.hv + h) * head;
    float4 s[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (row0 + i * RPW < a.dv) s[i] = ld_stream(&vec_at<const float4>(S, (int64_t)(row0 + i * RPW) * DK + col));
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      p[i] = 0.f;
      if (row0 + i * RPW < a.dv) {
        s[i].x = step(dec, s[i].x, v[i], k.x);
        s[i].y = step(dec, s[i].y, v[i], k.y);
        s[i].z = step(dec, s[i].z, v[i], k.z);
        s[i].w = step(dec, s[i].w, v[i], k.w);
        st_stream(&vec_at<float4>(S, (int64_t)(row0 + i * RPW) * DK + col), s[i]);
        p[i] = s[i].x * q.x + s[i].y * q.y + s[i].z * q.z + s[i].w * q.w;
      }
    }
  } else {
    if (cls == 2 && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
#pragma unroll
    for (int i = 0; i < NR; ++i) p[i] = 0.f;
  }
  // Sums over a row's lanes.  While a lane still holds several rows it gives
  // half of them to its partner: NR - 1 + log2(LPR / NR) exchanges for NR rows.
  int row = 0;  // among the thread's NR
  int o = LPR / 2;
#pragma unroll
  for (int n = NR; n > 1; n /= 2, o /= 2) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? p[i] : p[i + n / 2], keep = up ? p[i + n / 2] : p[i];
      p[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
    row += up ? n / 2 : 0;
  }
  const int writer = o;  // lanes whose remaining bits are zero write
#pragma unroll
  for (; o; o /= 2) p[0] += __shfl_xor_sync(0xffffffffu, p[0], o);
  const int at = row0 + row * RPW;
  if ((writer == 0 || (lane & (2 * writer - 1)) == 0) && at < a.dv) out[at] = from_f32<T>(p[0] * a.scale);
}

template <int DK, int NR, typename T>
cudaError_t decode_launch(const DecodeArgs& a, cudaStream_t s) {
  constexpr int per = kDT / 32 * (32 / (DK / 4)) * NR;
  return launch_pdl(lin_decode_kernel<DK, NR, T>, dim3((a.dv + per - 1) / per, a.hv, a.B), dim3(kDT), 0, s, dim3(1), a);
}

template <typename T>
cudaError_t decode_dispatch(const DecodeArgs& a, int dk, cudaStream_t s) {
  switch (dk) {
    case 16: return decode_launch<16, 1, T>(a, s);
    case 64: return decode_launch<64, 2, T>(a, s);
    case 128: return decode_launch<128, 4, T>(a, s);
  }
  return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// prefill, one token after another (every shape and type)
// ---------------------------------------------------------------------------
// A state row lies across DK / 16 lanes, 16 columns each (in runs of 4, so that
// the lanes' shared-memory accesses lie side by side), in registers; tokens
// come through shared memory in windows of up to 16, the next window's inputs
// requested a window ahead.  A window ends at a checkpoint.  Bound by issue: a
// token costs a warp 40 paired multiply-adds and 9 shared-memory reads for its 32
// x 16 values, 0.25 us with a CTA or two per SM; sequences are cut into segments
// to fill the SMs.
constexpr int kWin = 16;

__host__ __device__ constexpr int rec_min_threads(int dk) { return dk == 128 ? 128 : dk == 64 ? 64 : 32; }
// a thread per 16 columns of a row, a power of two of them, at most 256
int rec_threads(int dk, int dv) {
  int n = rec_min_threads(dk);
  while (n < 256 && n < dv * (dk / 16)) n *= 2;
  return n;
}

template <int DK, typename T, bool STATE>
__global__ void __launch_bounds__(256) lin_recurrent_kernel(const PrefillArgs a) {
  constexpr int LPR = DK / 16;
  // window elements per thread, at most (fewest threads)
  constexpr int QK = kWin * DK / rec_min_threads(DK), VV = kWin / LPR;
  extern __shared__ __align__(16) float smem[];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, nt = blockDim.x, R = nt / LPR, rsh = 31 - __clz(R);  // rows of a CTA: a power of two
  const int h = blockIdx.y;
  Segment s;
  if (!find_segment(a, blockIdx.z, s, tid == 0 && blockIdx.x == 0 && h == 0 && (!STATE))) return;
  if (STATE && (s.seg == s.n_seg - 1 || s.padded)) return;
  const int r0 = blockIdx.x * R, rows = min(R, a.dv - r0);
  const auto out = GDN_GV(reinterpret_cast<T*>(a.out), a.total * a.hv * a.dv);
  const int64_t ld = (int64_t)a.hv * a.dv;
  if (s.padded) {
    for (int64_t e = tid; e < (s.m1 - s.m0) * rows; e += nt)
      out[(s.t0 + s.m0 + e / rows) * ld + (int64_t)h * a.dv + r0 + e % rows] = from_f32<T>(0.f);
    return;
  }
  const auto sq = GDN_SV(smem, kWin * DK), sk = GDN_SV(smem + kWin * DK, kWin * DK);
  const auto sv = GDN_SV(smem + 2 * kWin * DK, kWin * R), so = GDN_SV(smem + 2 * kWin * DK + kWin * R, kWin * R);
  const auto x = GDN_GV(reinterpret_cast<const T*>(a.qkv), a.total * a.C);
  const int64_t kd = (int64_t)a.hk * DK, hq = h / a.G;
  const int row = tid / LPR, c0 = tid % LPR * 4;  // columns c0 + 4 LPR e, .. + 3 (e = 0 .. 3)
  const bool active = row < rows;
  const float ld_h = GDN_GV(a.log_decay, a.hv)[h];
  const Decay dec = decay_of(ld_h);
  const int64_t head = (int64_t)a.dv * DK, slot_n = a.hv * head;
  const int64_t own = h * head + (int64_t)(r0 + row) * DK + c0;  // this thread's place in a slot
  const auto pool = GDN_GV(a.ssm, a.num_slots * slot_n);
  const auto segs = GDN_GV(a.seg_state, a.n_segs * slot_n);
  float2 st[8];  // (pairs: two fused multiply-adds per instruction)
#pragma unroll
  for (int e = 0; e < 8; ++e) st[e] = make_float2(0.f, 0.f);
  if (active) {
    auto load = [&](const auto& from, Decay keep) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 u = vec_at<const float4>(from, own + 4 * LPR * e);
        st[2 * e] = add_decayed2(keep, st[2 * e], lo2(u));
        st[2 * e + 1] = add_decayed2(keep, st[2 * e + 1], hi2(u));
      }
    };
    const Decay none = {0.f, 0.f};
    if (s.seg == 0) {
      const bool kept = !STATE && s.n_seg > 1;
      if (kept) load(segs + (s.seg0 + s.n_seg - 1) * slot_n, none);
      else load(pool + (int64_t)s.slot * slot_n, none);
      if (STATE) {
        const auto keep = segs + (s.seg0 + s.n_seg - 1) * slot_n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vec_at<float4>(keep, own + 4 * LPR * e) = join4(st[2 * e], st[2 * e + 1]);
      }
    } else if (!STATE) {
      // the first segment's state holds the slot's already
      const Decay keep = decay_of(ld_h, (int64_t)s.chunks * kC);
      for (int k = 0; k < s.seg; ++k) load(segs + (s.seg0 + k) * slot_n, k ? keep : none);
    }
  }
  // the tokens until the next block boundary
  const int64_t blk = a.ckpt_block;
  int64_t bound = s.m0 + blk - (s.p0 + s.m0) % blk;  // tokens of the sequence up to it
  auto window = [&](int64_t m, int64_t bnd) { return (int)max((int64_t)0, min((int64_t)kWin, min(s.m1, bnd) - m)); };
  // A window's inputs as they are (a conversion beside its load would wait for
  // it, one load after another): of q and k this thread's column of every
  // (nt / DK)-th token, of v its row of every LPR-th.
  const int qc = tid % DK, qt = tid / DK, qstep = nt / DK, vr = tid & (R - 1), vt = tid >> rsh;
  T pq[QK], pk[QK], pv[VV];
  auto request = [&](int64_t m, int n) {
    const int64_t at = (s.t0 + m) * a.C;
    const auto xq = x + (at + hq * DK + qc), xv = x + (at + 2 * kd + (int64_t)h * a.dv + r0);
#pragma unroll
    for (int j = 0; j < QK; ++j) {
      const int t = qt + j * qstep;
      if (t < n) {
        if (!STATE) pq[j] = xq[t * a.C];
        pk[j] = xq[t * a.C + kd];
      }
    }
#pragma unroll
    for (int j = 0; j < VV; ++j) {
      const int t = vt + j * LPR;
      if (t < n && vr < rows) pv[j] = xv[t * a.C + vr];
    }
  };
  auto deposit = [&](int n) {
#pragma unroll
    for (int j = 0; j < QK; ++j) {
      const int t = qt + j * qstep;
      if (t < n) {
        if (!STATE) sq[t * DK + qc] = to_f32(pq[j]);
        sk[t * DK + qc] = to_f32(pk[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < VV; ++j) {
      const int t = vt + j * LPR;
      if (t < n) sv[(t << rsh) + vr] = vr < rows ? to_f32(pv[j]) : 0.f;
    }
  };
  int64_t m = s.m0;
  int n = window(m, bound);
  request(m, n);
  while (n > 0) {
    deposit(n);
    __syncthreads();
    const bool at_bound = m + n == bound;
    const int64_t mb = at_bound ? bound + blk : bound;
    const int nn = window(m + n, mb);
    if (nn > 0) request(m + n, nn);
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      const float v = sv[(t << rsh) + row];
      float2 p[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 k4 = vec_at<const float4>(sk, t * DK + c0 + 4 * LPR * e);
        st[2 * e] = step2(dec, st[2 * e], v, lo2(k4));
        st[2 * e + 1] = step2(dec, st[2 * e + 1], v, hi2(k4));
        if (!STATE) {
          const float4 q4 = vec_at<const float4>(sq, t * DK + c0 + 4 * LPR * e);
          p[0] = fma2(st[2 * e], lo2(q4), p[0]);
          p[1] = fma2(st[2 * e + 1], hi2(q4), p[1]);
        }
      }
      if (!STATE) {
        float o = (p[0].x + p[0].y) + (p[1].x + p[1].y);
#pragma unroll
        for (int w = LPR / 2; w; w /= 2) o += __shfl_xor_sync(0xffffffffu, o, w);
        if (active && tid % LPR == 0) so[(t << rsh) + row] = o * a.scale;
      }
    }
    auto store = [&](const auto& to) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        vec_at<float4>(to, own + 4 * LPR * e) = join4(st[2 * e], st[2 * e + 1]);
    };
    if (!STATE && at_bound && active) {
      const int64_t idx = bound + s.p0;  // the boundary's position
      const int64_t i = idx / blk - s.p0 / blk - 1;
      if (i < a.max_ckpt) {
        const int32_t id = GDN_GV(a.ckpt_ids, (long long)a.n_seq * a.max_ckpt)[(int64_t)s.n * a.max_ckpt + i];
        const int cls = slot_class(id, a.ck_num_slots);
        if (cls == 0) store(GDN_GV(a.ck_ssm, a.ck_num_slots * slot_n) + (int64_t)id * slot_n);
        else if (cls == 2) report(a.err, GDN_DEV_ERR_SLOT_OOB);
      }
    }
    __syncthreads();  // so complete; q, k, v may be replaced
    if (!STATE)
      for (int e = tid; e < n << rsh; e += nt)
        if ((e & (R - 1)) < rows)
          out[(s.t0 + m + (e >> rsh)) * ld + (int64_t)h * a.dv + r0 + (e & (R - 1))] = from_f32<T>(so[e]);
    m += n;
    n = nn;
    bound = mb;
    // the last segment's state replaces the slot's: the second launch reads
    // no slot that has several segments
    if (n <= 0 && active) {
      if (STATE) store(segs + (s.seg0 + s.seg) * slot_n);
      else if (s.seg == s.n_seg - 1) store(pool + (int64_t)s.slot * slot_n);
    }
    if (!STATE) __syncthreads();  // so read before the next window's outputs
  }
}

template <int DK, typename T>
cudaError_t recurrent_launch(const PrefillArgs& a, cudaStream_t s) {
  constexpr int LPR = DK / 16;
  const int nt = rec_threads(DK, a.dv), R = nt / LPR;
  const size_t smem = sizeof(float) * (2 * kWin * DK + 2 * kWin * (size_t)R);
  const dim3 grid((a.dv + R - 1) / R, a.hv, a.n_segs);
  if (a.seg_state) {
    const cudaError_t e = launch_pdl(lin_recurrent_kernel<DK, T, true>, grid, dim3(nt), smem, s, dim3(1), a);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(lin_recurrent_kernel<DK, T, false>, grid, dim3(nt), smem, s, dim3(1), a);
}

template <typename T>
cudaError_t recurrent_dispatch(const PrefillArgs& a, cudaStream_t s) {
  switch (a.dk) {
    case 16: return recurrent_launch<16, T>(a, s);
    case 64: return recurrent_launch<64, T>(a, s);
    case 128: return recurrent_launch<128, T>(a, s);
  }
  return cudaErrorInvalidValue;
}

// Blocks per segment (kWhole: sequences stay whole).  The lengths are on the
// device: the rule sees their number and sum.
// Chunk form, one CTA per head and segment on an SM, some 1.75 us a block, and
// 0.72 us in the state pass before it: segments of the length at which all of
// them are one wave on the SMs, not below kMinSeg blocks.  Flags, another launch
// and joining the states (a segment reads all its predecessors') cost some 6 us:
// worth it if the longest sequence takes longer whole,
//   1.75 longest > (1.75 + 0.72) segment + 6,
// which the device decides where it is not known here.  Measured with 32 heads, cut
// and whole: 8192 tokens 92 and 217 us, 5000 + 1000 + 1000 87 and 136, 2 x 2048 51
// and 60; 3 x 2700 90 and 78 (two waves), 2 x 1024 36 and 34.
constexpr int64_t kMinSeg = 8, kMaxSegs = 16;
int64_t cut_from(int64_t seg) { return (10 * seg + 24) / 7 + 1; }
int64_t chunk_seg(const gdn_dims& d, int32_t n_seq, int64_t total) {
  const int64_t chunks = (total + kC - 1) / kC, mean = (chunks + n_seq - 1) / n_seq, wave = sm_count() / d.hv;
  if (wave < 2 || n_seq > kMaxCut) return kWhole;
  // (a sequence's blocks may be one more than its length says.)  First segments run
  // beside the state pass on the SMs that it leaves free.  Where those are half
  // of the heads or more, the blocks are divided by 0.45 of a wave more: with 0, 0.25
  // and 0.45 of one, 32 heads, 8192 tokens 98, 96 and 92 us, 6000 + 2000 95, 93 and 90,
  // 5000 + 1000 + 1000 90, 88 and 87; 20 heads, 8192 tokens 70, 68 and 68; 16 heads 60,
  // 59 and 59.  (48 and 64 heads leave too few; one 0.45 for all numbers of heads.)
  const int64_t spare = 2 * (sm_count() - wave * d.hv) >= d.hv ? 45 : 0, all = 100 * (chunks + n_seq - 1);
  const int64_t seg = std::max(std::max((all + 100 * wave + spare - 1) / (100 * wave + spare) + 1, kMinSeg),
                               (mean + kMaxSegs - 1) / kMaxSegs);
  return chunks < cut_from(seg) ? kWhole : seg;
}
// Recurrence, a block in some 16 us and 10 in the state pass: as short segments
// as give 3 CTAs per SM, at most kMaxRecSegs per sequence of the mean length; a
// mean below two segments stays whole.  Cut and whole, 16 heads of 64 x 64: 1024
// tokens 46 and 278 us (in segments of 2 blocks 79), 2048 tokens 85 (2 blocks; of 1
// block 91) and 553; 8 x 60 tokens 30 and 20.
constexpr int64_t kMaxRecSegs = 32;
int64_t rec_seg(const gdn_dims& d, int32_t n_seq, int64_t total) {
  const int64_t chunks = (total + kC - 1) / kC, mean = (chunks + n_seq - 1) / n_seq;
  const int64_t rows = rec_threads(d.dk, d.dv) / (d.dk / 16), ctas = d.hv * ((d.dv + rows - 1) / rows);
  const int64_t fill = 3LL * sm_count();
  const int64_t seg = std::max(((chunks + n_seq) * ctas + fill - 1) / fill, (mean + kMaxRecSegs - 1) / kMaxRecSegs);
  return mean < 2 * seg ? kWhole : seg;
}
int64_t seg_chunks(const gdn_dims& d, int32_t n_seq, int64_t total, bool chunked) {
  return chunked ? chunk_seg(d, n_seq, total) : rec_seg(d, n_seq, total);
}
int64_t seg_slots(int64_t sc, int32_t n_seq, int64_t total) { return first_slot(total, n_seq) / sc + n_seq; }

gdn_status check_lin(const gdn_dims* d) {
  const gdn_status st = check_dims_state(d);
  if (st != GDN_OK) return st;
  if (d->conv_width != 1) return GDN_ERR_UNSUPPORTED;
  return d->hv > 65535 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_lin_decode_step(const gdn_dims* dims, gdn_pool pool, const float* log_decay, float scale,
                                          const int32_t* slot_ids, int32_t B, const void* qkv, void* out,
                                          uint32_t* dev_err, void* stream) {
  using namespace gdn;
  gdn_status st = check_lin(dims);
  if (st != GDN_OK) return st;
  if (B < 0) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if (B > 65535) return GDN_ERR_UNSUPPORTED;
  if ((st = check_pool(*dims, pool)) != GDN_OK) return st;
  if (!log_decay || !slot_ids || !qkv || !out) return GDN_ERR_INVALID_ARG;
  DecodeArgs a = {};
  a.ssm = pool.ssm;
  a.num_slots = pool.num_slots;
  a.log_decay = log_decay;
  a.scale = scale;
  a.slot_ids = slot_ids;
  a.qkv = qkv;
  a.out = out;
  a.err = dev_err;
  a.B = B;
  a.hk = dims->hk;
  a.hv = dims->hv;
  a.dv = dims->dv;
  a.G = dims->hv / dims->hk;
  a.C = channels(*dims);
  const size_t e4 = 4 * dtype_size(dims->act_dtype);
  a.vec = a.C % 4 == 0 && aligned(qkv, e4);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dims->act_dtype == GDN_BF16 ? decode_dispatch<__nv_bfloat16>(a, dims->dk, s)
                                                    : decode_dispatch<float>(a, dims->dk, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_LIN_DECODE);
  return GDN_OK;
}

extern "C" size_t gdn_lin_prefill_workspace_size(const gdn_dims* dims, int32_t n_seq, int64_t total_tokens) {
  using namespace gdn;
  if (check_lin(dims) != GDN_OK || n_seq <= 0 || total_tokens <= 0) return 0;
  // (which form runs depends on the tensors' alignment, too)
  size_t most = 0;
  for (int chunked = 0; chunked <= (lin::chunk_shape(*dims) ? 1 : 0); ++chunked) {
    const int64_t sc = seg_chunks(*dims, n_seq, total_tokens, chunked), segs = seg_slots(sc, n_seq, total_tokens);
    if (sc < lin::first_slot(total_tokens, n_seq))
      most = std::max(most, (size_t)segs * ssm_slot_bytes(*dims) + (chunked ? 4 * lin::sync_words(segs, dims->hv) : 0));
  }
  return most;
}

extern "C" gdn_status gdn_lin_prefill(const gdn_dims* dims, gdn_pool pool, gdn_pool ckpt, const float* log_decay,
                                      float scale, const int32_t* slot_ids, const int32_t* cu_seqlens,
                                      const int64_t* start_pos, int32_t n_seq, int64_t total_tokens,
                                      const int32_t* ckpt_ids, int32_t max_ckpt, int32_t ckpt_block, const void* qkv,
                                      void* out, void* workspace, size_t workspace_bytes, uint32_t* dev_err,
                                      void* stream) {
  using namespace gdn;
  gdn_status st = check_lin(dims);
  if (st != GDN_OK) return st;
  if (n_seq < 0 || total_tokens < 0 || max_ckpt < 0) return GDN_ERR_INVALID_ARG;
  if (ckpt_block <= 0 || ckpt_block % lin::kC) return GDN_ERR_INVALID_ARG;
  if (n_seq == 0) return GDN_OK;
  if (n_seq > 16384 || total_tokens > 2147483647LL) return GDN_ERR_UNSUPPORTED;
  if ((st = check_pool(*dims, pool)) != GDN_OK) return st;
  if (max_ckpt > 0 && (st = check_pool(*dims, ckpt)) != GDN_OK) return st;
  if (!log_decay || !slot_ids || !cu_seqlens || !start_pos || (max_ckpt > 0 && !ckpt_ids)) return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!qkv || !out)) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_lin_prefill_workspace_size(dims, n_seq, total_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return GDN_ERR_INVALID_ARG;
  lin::PrefillArgs a = {};
  a.ssm = pool.ssm;
  a.num_slots = pool.num_slots;
  a.ck_ssm = ckpt.ssm;
  a.ck_num_slots = max_ckpt > 0 ? ckpt.num_slots : 0;
  a.log_decay = log_decay;
  a.scale = scale;
  a.slot_ids = slot_ids;
  a.cu_seqlens = cu_seqlens;
  a.start_pos = start_pos;
  a.n_seq = n_seq;
  a.total = total_tokens;
  a.ckpt_ids = ckpt_ids;
  a.max_ckpt = max_ckpt;
  a.ckpt_block = ckpt_block;
  a.qkv = qkv;
  a.out = out;
  a.err = dev_err;
  a.hk = dims->hk;
  a.hv = dims->hv;
  a.dk = dims->dk;
  a.dv = dims->dv;
  a.G = dims->hv / dims->hk;
  a.C = channels(*dims);
  // GDN_LIN_PREFILL_PATH=recurrent (read on every call) forces the recurrence
  const char* path = std::getenv("GDN_LIN_PREFILL_PATH");
  const bool chunked = lin::chunk_supported(*dims, total_tokens, qkv, out) && !(path && !std::strcmp(path, "recurrent"));
  const int64_t sc = seg_chunks(*dims, n_seq, total_tokens, chunked), segs = seg_slots(sc, n_seq, total_tokens);
  if (segs > 65535) return GDN_ERR_UNSUPPORTED;
  a.seg_chunks = (int32_t)sc;
  a.n_segs = (int32_t)segs;
  a.seg_state = sc < lin::first_slot(total_tokens, n_seq) ? reinterpret_cast<float*>(workspace) : nullptr;
  if (chunked && a.seg_state) {
    a.sync = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + (size_t)segs * ssm_slot_bytes(*dims));
    a.cut_from = (int32_t)std::min<int64_t>(cut_from(sc), INT32_MAX);
    // a sequence of b blocks has (b - 1) / sc segments beyond its first one, and all
    // have at most total / 64 + 2 n_seq blocks
    a.max_extra = (int32_t)((total_tokens / lin::kC + n_seq) / sc);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = chunked                          ? lin::chunk_launch(a, s)
                        : dims->act_dtype == GDN_BF16 ? recurrent_dispatch<__nv_bfloat16>(a, s)
                                                      : recurrent_dispatch<float>(a, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_LIN_PREFILL);
  return GDN_OK;
}
