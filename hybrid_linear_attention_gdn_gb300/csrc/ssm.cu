// Selective state space step over the slot pool (Gu & Dao, "Mamba", 2023;
// Dao & Gu, "Transformers are SSMs", ICML 2024; the pages name the family in
// TokenSpeed Qwen3.5 page, "Prefix cache para arquitecturas GDN/Mamba"):
//   y = SiLU(conv1d(history, x) + bias);  q, k, v = split(y)
//   dt = softplus(a + dt_bias);  S <- exp(-exp(A_log) dt) S + dt k v^T
//   o = S^T q + D v
// Here: the decode step, and the token recurrence of the prefill for the
// shapes that its chunked form does not take.
#include "ssm.cuh"
#include "ssm_chunk.cuh"
#include "decode_tma.cuh"  // sm_count
#include "prefill_tc.cuh"  // conv_history_launch

#include <cstring>

namespace gdn {
namespace {

using namespace ssm;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// A state row of DK floats is DK / 4 lanes of one float4; a warp-wide access
// covers RPW rows.
template <int DK>
struct Rows {
  static constexpr int LPR = DK / 4;    // lanes per row
  static constexpr int RPW = 32 / LPR;  // rows per warp-wide access
};

// Sums of UN values over the LPR lanes of a row, transposed: each exchange
// halves the values a lane still carries, so UN sums cost about UN + log2(LPR)
// shuffles instead of UN log2(LPR).  Afterwards the lane holds
// max(1, UN / LPR) complete sums in o[0 ..]; o[i] belongs to value u + i,
// where u is the return value, and when UN < LPR the lanes with writer set
// hold each sum once.
template <int UN, int LPR>
__device__ __forceinline__ int reduce_rows(float (&o)[UN], bool& writer) {
  const int lane = threadIdx.x & 31;
  int u = 0, cnt = UN;
  writer = true;
#pragma unroll
  for (int m = LPR / 2; m >= 1; m >>= 1) {
    const bool up = (lane & m) != 0;
    if (cnt > 1) {
      cnt >>= 1;
#pragma unroll
      for (int i = 0; i < UN / 2; ++i) {
        if (i < cnt) {
          const float keep = up ? o[i + cnt] : o[i], give = up ? o[i] : o[i + cnt];
          o[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
      }
      u += up ? cnt : 0;
    } else {
      o[0] += __shfl_xor_sync(0xffffffffu, o[0], m);
      writer = writer && !up;
    }
  }
  return u;
}

// ---------------------------------------------------------------------------
// decode
// ---------------------------------------------------------------------------
// The split form, for few requests and for shapes that the persistent form
// (ssm_ring.cu) does not take.
// HBM bound: the state is read and written once (8 dk bytes per row), all
// else is about 1 % of it.  A cluster of `cs` CTAs takes one request and one
// QK head hq: the G dv state rows of the V heads that read hq are split
// evenly over the CTAs, each of which computes the q and k features itself.
// The cluster exists for the conv history: q and k inputs are read by every
// CTA, so the first one shifts them only after the cluster's barrier, which
// every CTA reaches long before the first has streamed its rows.  Each warp
// holds UN accesses of rows in flight, the first batch requested before the
// features are computed; several CTAs per SM cover one another's prologues.
// 64 heads of 64 in 8 groups, graph of calls: 1 / 4 / 24 requests 5.0 / 8.2 /
// 21.4 us (0.12 / 0.30 / 0.69 of the copy bandwidth); 32 heads of 64 in one
// group, 64 / 256 requests 29.8 / 98 us (0.66 / 0.81).
template <int DK, int UN, typename Tact, typename Tconv>
__global__ void __launch_bounds__(kThreads, 3) ssm_decode_kernel(const DecodeArgs a) {
  using M = Rows<DK>;
  static_assert(2 * DK <= kThreads, "one q or k channel per thread");
  extern __shared__ __align__(16) float smem[];
  const auto sqk = GDN_SV(smem, 2 * DK);                 // q, k
  const auto sdx = GDN_SV(smem + 2 * DK, a.rpc);         // dt v per row
  const auto sal = GDN_SV(smem + 2 * DK + a.rpc, a.rpc);  // alpha per row
  const auto sdv = GDN_SV(smem + 2 * DK + 2 * a.rpc, a.rpc);  // D v per row
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.y, hq = blockIdx.x / a.cs, rank = blockIdx.x % a.cs;
  const int lo = rank * a.rpc, hi = min(a.G * a.dv, lo + a.rpc);  // rows of the group
  const auto out = GDN_GV(reinterpret_cast<Tact*>(a.out), (long long)a.B * a.hv * a.dv);
  const size_t out0 = ((size_t)r * a.hv + (size_t)hq * a.G) * a.dv;
  const int32_t slot = GDN_GV(a.slot_ids, a.B)[r];
  const int cls = slot_class(slot, a.num_slots);
  if (cls) {  // the same in every CTA of the cluster
    if (cls == 2 && blockIdx.x == 0 && tid == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
    for (int i = lo + tid; i < hi; i += kThreads) out[out0 + i] = from_f32<Tact>(0.f);
    return;
  }
  const auto S = GDN_GV(a.ssm, (long long)a.num_slots * a.hv * a.dv * DK) +
                 ((size_t)slot * a.hv + (size_t)hq * a.G) * a.dv * DK;
  const int sub = lane / M::LPR, seg = lane % M::LPR;
  constexpr int kWarpRows = UN * M::RPW, kBatch = kWarps * kWarpRows;
  int row = lo + warp * kWarpRows + sub;  // this lane's row of access u: row + u * RPW
  float4 s[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (row + u * M::RPW < hi)
      s[u] = ld_stream(&vec_at<const float4>(S, (size_t)(row + u * M::RPW) * DK + 4 * seg));
  // features: conv1d over the history and the new input, SiLU
  const auto hist = GDN_GV(reinterpret_cast<Tconv*>(a.conv), (long long)a.num_slots * (a.W - 1) * a.C) +
                    (size_t)slot * (a.W - 1) * a.C;
  const auto x = GDN_GV(reinterpret_cast<const Tact*>(a.qkv), (long long)a.B * a.C) + (size_t)r * a.C;
  const auto conv_w = GDN_GV(a.conv_w, (long long)a.C * a.W);
  Tconv win[kMaxW];  // taps 0 .. W - 1 of a channel, oldest first
  auto feature = [&](int c) -> float {
    float acc = a.conv_bias ? GDN_GV(a.conv_bias, a.C)[c] : 0.f;
#pragma unroll
    for (int j = 0; j < kMaxW; ++j)
      if (j < a.W) {
        const float v = j < a.W - 1 ? to_f32(win[j] = hist[(size_t)j * a.C + c]) : to_f32(x[c]);
        acc = fmaf(conv_w[(size_t)c * a.W + j], v, acc);
        if (j == a.W - 1) win[j] = from_f32<Tconv>(v);
      }
    return silu_f(acc);
  };
  auto shift = [&](int c) {  // the history after this token
#pragma unroll
    for (int j = 0; j < kMaxW - 1; ++j)
      if (j < a.W - 1) hist[(size_t)j * a.C + c] = win[j + 1];
  };
  const auto gate_a = GDN_GV(reinterpret_cast<const Tact*>(a.a), (long long)a.B * a.hv);
  for (int i = lo + tid; i < hi; i += kThreads) {
    const int h = hq * a.G + i / a.dv, c = 2 * a.hk * DK + hq * a.G * a.dv + i;
    const float v = feature(c);
    shift(c);
    const Gate g = gate(GDN_GV(a.A_log, a.hv)[h], GDN_GV(a.dt_bias, a.hv)[h],
                        to_f32(gate_a[(size_t)r * a.hv + h]));
    sdx[i - lo] = g.dt * v;
    sal[i - lo] = expf(g.g);
    sdv[i - lo] = a.D ? GDN_GV(a.D, a.hv)[h] * v : 0.f;
  }
  const int cqk = (tid < DK ? hq * DK : (a.hk + hq - 1) * DK) + tid;
  if (tid < 2 * DK) sqk[tid] = feature(cqk);
  if (a.cs > 1) cluster_arrive_release();
  __syncthreads();
  if (a.cs == 1 && tid < 2 * DK) shift(cqk);
  const float4 q4 = vec_at<const float4>(sqk, 4 * seg), k4 = vec_at<const float4>(sqk, DK + 4 * seg);
  for (int r0 = lo; r0 < hi; r0 += kBatch, row += kBatch) {
    float o[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      o[u] = 0.f;
      const int i = row + u * M::RPW;
      if (i < hi) {
        const float al = sal[i - lo], dx = sdx[i - lo];
        s[u].x = fmaf(dx, k4.x, al * s[u].x);
        s[u].y = fmaf(dx, k4.y, al * s[u].y);
        s[u].z = fmaf(dx, k4.z, al * s[u].z);
        s[u].w = fmaf(dx, k4.w, al * s[u].w);
        st_stream(&vec_at<float4>(S, (size_t)i * DK + 4 * seg), s[u]);
        o[u] = s[u].x * q4.x + s[u].y * q4.y + s[u].z * q4.z + s[u].w * q4.w;
        if (i + kBatch < hi) s[u] = ld_stream(&vec_at<const float4>(S, (size_t)(i + kBatch) * DK + 4 * seg));
      }
    }
    bool writer;
    const int u0 = reduce_rows<UN, M::LPR>(o, writer);
#pragma unroll
    for (int k = 0; k < (UN > M::LPR ? UN / M::LPR : 1); ++k) {
      const int i = row + (u0 + k) * M::RPW;
      if (writer && i < hi) out[out0 + i] = from_f32<Tact>(o[k] + sdv[i - lo]);
    }
  }
  if (a.cs > 1) {
    cluster_wait_acquire();
    if (rank == 0 && tid < 2 * DK) {
      shift(cqk);
    }
  }
}

template <int DK, int UN, typename Tact, typename Tconv>
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s) {
  const size_t smem = (2 * DK + 3 * (size_t)a.rpc) * sizeof(float);
  return launch_pdl(ssm_decode_kernel<DK, UN, Tact, Tconv>, dim3((unsigned)(a.hk * a.cs), (unsigned)a.B),
                    dim3(kThreads), smem, s, dim3((unsigned)a.cs), a);
}

template <int DK, int UN>
cudaError_t dispatch_decode(const DecodeArgs& a, int act, int cv, cudaStream_t s) {
  if (act == GDN_F32) return launch_decode<DK, UN, float, float>(a, s);
  if (cv == GDN_BF16) return launch_decode<DK, UN, __nv_bfloat16, __nv_bfloat16>(a, s);
  return launch_decode<DK, UN, __nv_bfloat16, float>(a, s);
}

// ---------------------------------------------------------------------------
// prefill, token recurrence
// ---------------------------------------------------------------------------
// For the shapes that the chunked form does not take.  A CTA owns up to
// kWarps UN RPW state rows of one V head of one sequence and keeps them in
// registers from the first token to the last; windows of kTW tokens'
// features and gates are computed into shared memory, then every warp walks
// the window's tokens on its rows.  Bound by the latency of a token's chain
// (update, dot product, transposed reduction), not by memory.  Measured: 513
// tokens of 32 heads of 64 x 128 240 us in a graph, 0.47 us a token (84 us more
// without a window's inputs requested a window ahead, 26 more with eight taps
// for a conv of four); 233 tokens of the smallest layer 49 us.  The checkpoint
// test taken out of the token loop and unrolling it by 2 to 8 changed nothing
// or cost up to 9 %.
constexpr int kTW = 16;

// SiLU as x e^min(x, 0) / (1 + e^-|x|), to some 3 units in the last place (6 at
// most) for x >= -87; below, where the exponential leaves the normal range, to
// 90 2^-126.  The exponential is at most 1, so nothing overflows: it is
// 2^(-|x| log2 e) with what the product lost put back (|x| held at 127, where
// it is 0, so that what was lost is finite); the quotient is approximate.  An
// infinity or a NaN gives what x / (1 + e^-x) gives.  Its rms error is 1.2 times
// that of the library's exponential and division, with which 513 tokens of 32
// heads of 64 x 128 take 280 us, not 240, and the fp32 outputs' error against
// float64 is 0 to 7 % smaller.
__device__ __forceinline__ float silu_approx(float x) {
  const float c = fminf(fabsf(x), 127.f);
  const float t = c * -1.44269504f, lost = fmaf(c, -1.92596299e-8f, fmaf(c, -1.44269504f, -t));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(t));
  e = fmaf(e, lost * 0.693147181f, e);
  return __fdividef(x < 0.f ? x * e : x, 1.f + e);
}

template <int DK, int UN, int TAPS, typename Tact, typename Tconv>
__global__ void __launch_bounds__(kThreads) ssm_recurrent_kernel(const PrefillArgs a, const int parts) {
  using M = Rows<DK>;
  constexpr int kWarpRows = UN * M::RPW, R = kWarps * kWarpRows, NCH = 2 * DK + R;
  constexpr int kCPT = (NCH + kThreads - 1) / kThreads;  // channels per thread
  __shared__ __align__(16) float sy_[kTW][NCH];
  __shared__ float so_[kTW][R];
  __shared__ float sal_[kTW], sdt_[kTW];
  const auto sy = GDN_SV(&sy_[0][0], kTW * NCH);
  const auto so = GDN_SV(&so_[0][0], kTW * R);
  const auto sal = GDN_SV(sal_, kTW), sdt = GDN_SV(sdt_, kTW);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = blockIdx.y, h = blockIdx.x / parts, hq = h / a.G, row0 = (blockIdx.x % parts) * R;
  const int nrows = min(R, a.dv - row0);
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  const int64_t t0 = cu[n], len = (int64_t)cu[n + 1] - t0, p0 = GDN_GV(a.start_pos, a.n_seq)[n];
  if (t0 < 0 || len < 0 || t0 + len > a.total || p0 < 0) {
    if (blockIdx.x == 0 && tid == 0) report(a.err, GDN_DEV_ERR_SEQLENS);
    return;
  }
  const auto out = GDN_GV(reinterpret_cast<Tact*>(a.out), a.total * a.hv * a.dv);
  const int32_t slot = GDN_GV(a.slot_ids, a.n_seq)[n];
  const int cls = slot_class(slot, a.num_slots);
  if (cls) {
    if (cls == 2 && blockIdx.x == 0 && tid == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
    for (int64_t e = tid; e < len * nrows; e += kThreads)
      out[((t0 + e / nrows) * a.hv + h) * a.dv + row0 + e % nrows] = from_f32<Tact>(0.f);
    return;
  }
  if (len == 0) return;
  const long long state = (long long)a.hv * a.dv * DK;
  const auto S = GDN_GV(a.ssm, a.num_slots * state) + (((size_t)slot * a.hv + h) * a.dv + row0) * DK;
  const auto qkv = GDN_GV(reinterpret_cast<const Tact*>(a.qkv), a.total * a.C);
  const auto gate_a = GDN_GV(reinterpret_cast<const Tact*>(a.a), a.total * a.hv);
  const int sub = lane / M::LPR, seg = lane % M::LPR;
  const int row = warp * kWarpRows + sub;
  float4 s[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    s[u] = row + u * M::RPW < nrows ? vec_at<const float4>(S, (size_t)(row + u * M::RPW) * DK + 4 * seg)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
  // this thread's channels: weights and history right-aligned in TAPS taps
  float w[kCPT][TAPS], win[kCPT][TAPS - 1], bias[kCPT];
  int ch[kCPT];
  const int lead = TAPS - a.W;
  const auto hist = GDN_GV(reinterpret_cast<const Tconv*>(a.conv), (long long)a.num_slots * (a.W - 1) * a.C) +
                    (size_t)slot * (a.W - 1) * a.C;
  const auto conv_w = GDN_GV(a.conv_w, (long long)a.C * a.W);
#pragma unroll
  for (int ci = 0; ci < kCPT; ++ci) {
    const int i = tid + ci * kThreads;
    ch[ci] = i < DK ? hq * DK + i
             : i < 2 * DK ? (a.hk + hq) * DK + (i - DK)
             : i < 2 * DK + nrows ? 2 * a.hk * DK + h * a.dv + row0 + (i - 2 * DK)
                                  : -1;
    if (ch[ci] < 0) continue;
    bias[ci] = a.conv_bias ? GDN_GV(a.conv_bias, a.C)[ch[ci]] : 0.f;
#pragma unroll
    for (int j = 0; j < TAPS; ++j) w[ci][j] = j >= lead ? conv_w[(size_t)ch[ci] * a.W + (j - lead)] : 0.f;
#pragma unroll
    for (int j = 0; j < TAPS - 1; ++j) win[ci][j] = j >= lead ? to_f32(hist[(size_t)(j - lead) * a.C + ch[ci]]) : 0.f;
  }
  const float A_log = GDN_GV(a.A_log, a.hv)[h], dtb = GDN_GV(a.dt_bias, a.hv)[h];
  const float D = a.D ? GDN_GV(a.D, a.hv)[h] : 0.f;
  const int64_t blk0 = p0 / a.ckpt_block;
  int64_t next_bd = (blk0 + 1) * a.ckpt_block, ck_idx = 0;

  // a window's inputs, requested while the one before it is walked
  Tact xv[kCPT][kTW], ga = {};
  auto request = [&](int64_t w0) {
#pragma unroll
    for (int ci = 0; ci < kCPT; ++ci)
#pragma unroll
      for (int t = 0; t < kTW; ++t)
        xv[ci][t] = ch[ci] >= 0 && w0 + t < len ? qkv[(size_t)(t0 + w0 + t) * a.C + ch[ci]] : from_f32<Tact>(0.f);
    if (tid < kTW && w0 + tid < len) ga = gate_a[(size_t)(t0 + w0 + tid) * a.hv + h];
  };
  request(0);
  for (int64_t w0 = 0; w0 < len; w0 += kTW) {
    const int nt = len - w0 < kTW ? (int)(len - w0) : kTW;
#pragma unroll
    for (int ci = 0; ci < kCPT; ++ci) {
      if (ch[ci] < 0) continue;
#pragma unroll
      for (int t = 0; t < kTW; ++t) {
        float acc = bias[ci];
#pragma unroll
        for (int j = 0; j < TAPS - 1; ++j) acc = fmaf(w[ci][j], win[ci][j], acc);
        const float x = to_f32(xv[ci][t]);
        acc = fmaf(w[ci][TAPS - 1], x, acc);
        sy[t * NCH + tid + ci * kThreads] = silu_approx(acc);
        // (past the end, in a last window, nothing reads these)
#pragma unroll
        for (int j = 0; j < TAPS - 2; ++j) win[ci][j] = win[ci][j + 1];
        win[ci][TAPS - 2] = x;
      }
    }
    if (tid < nt) {
      const Gate g = gate(A_log, dtb, to_f32(ga));
      sal[tid] = expf(g.g);
      sdt[tid] = g.dt;
    }
    __syncthreads();
    request(w0 + kTW);
    for (int t = 0; t < nt; ++t) {
      const auto y = sy + t * NCH;
      const float4 q4 = vec_at<const float4>(y, 4 * seg), k4 = vec_at<const float4>(y, DK + 4 * seg);
      const float al = sal[t], dt = sdt[t];
      float o[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = row + u * M::RPW;
        const float dx = i < nrows ? dt * y[2 * DK + i] : 0.f;
        s[u].x = fmaf(dx, k4.x, al * s[u].x);
        s[u].y = fmaf(dx, k4.y, al * s[u].y);
        s[u].z = fmaf(dx, k4.z, al * s[u].z);
        s[u].w = fmaf(dx, k4.w, al * s[u].w);
        o[u] = s[u].x * q4.x + s[u].y * q4.y + s[u].z * q4.z + s[u].w * q4.w;
      }
      bool writer;
      const int u0 = reduce_rows<UN, M::LPR>(o, writer);
#pragma unroll
      for (int k = 0; k < (UN > M::LPR ? UN / M::LPR : 1); ++k) {
        const int i = row + (u0 + k) * M::RPW;
        if (writer && i < nrows) so[t * R + i] = o[k] + D * y[2 * DK + i];
      }
      if (p0 + w0 + t + 1 == next_bd) {
        if (ck_idx < a.max_ckpt) {
          const int32_t cid = GDN_GV(a.ckpt_ids, (long long)a.n_seq * a.max_ckpt)[(size_t)n * a.max_ckpt + ck_idx];
          if (slot_class(cid, a.ck_num_slots) == 0) {
            const auto K = GDN_GV(a.ck_ssm, a.ck_num_slots * state) + (((size_t)cid * a.hv + h) * a.dv + row0) * DK;
#pragma unroll
            for (int u = 0; u < UN; ++u)
              if (row + u * M::RPW < nrows) vec_at<float4>(K, (size_t)(row + u * M::RPW) * DK + 4 * seg) = s[u];
          }
        }
        ++ck_idx;
        next_bd += a.ckpt_block;
      }
    }
    __syncthreads();
    for (int e = tid; e < nt * nrows; e += kThreads)
      out[((size_t)(t0 + w0 + e / nrows) * a.hv + h) * a.dv + row0 + e % nrows] =
          from_f32<Tact>(so[(e / nrows) * R + e % nrows]);
  }
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (row + u * M::RPW < nrows) vec_at<float4>(S, (size_t)(row + u * M::RPW) * DK + 4 * seg) = s[u];
}

template <int DK, int UN, int TAPS>
cudaError_t launch_recurrent(const PrefillArgs& a, int act, int cv, cudaStream_t s) {
  constexpr int R = kWarps * UN * Rows<DK>::RPW;
  const int parts = (a.dv + R - 1) / R;
  const dim3 grid((unsigned)(a.hv * parts), (unsigned)a.n_seq), block(kThreads);
  using B = __nv_bfloat16;
  if (act == GDN_F32)
    return launch_plain(ssm_recurrent_kernel<DK, UN, TAPS, float, float>, grid, block, 0, s, dim3(1), a, parts);
  if (cv == GDN_BF16)
    return launch_plain(ssm_recurrent_kernel<DK, UN, TAPS, B, B>, grid, block, 0, s, dim3(1), a, parts);
  return launch_plain(ssm_recurrent_kernel<DK, UN, TAPS, B, float>, grid, block, 0, s, dim3(1), a, parts);
}
template <int DK, int UN>
cudaError_t dispatch_recurrent(const PrefillArgs& a, int act, int cv, cudaStream_t s) {
  return a.W <= 4 ? launch_recurrent<DK, UN, 4>(a, act, cv, s) : launch_recurrent<DK, UN, kMaxW>(a, act, cv, s);
}

gdn_status check_params(const gdn_ssm_params* p) {
  if (!p || !p->conv_w || !p->A_log || !p->dt_bias) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_ssm_decode_step(const gdn_dims* dims, gdn_pool pool, const gdn_ssm_params* params,
                                          const int32_t* slot_ids, int32_t B, const void* qkv, const void* a,
                                          void* out, uint32_t* dev_err, void* stream) {
  using namespace gdn;
  gdn_status st = check_dims(dims);
  if (st != GDN_OK) return st;
  if (B < 0) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  const int64_t rows = (int64_t)(dims->hv / dims->hk) * dims->dv;
  if (B > 65535 || rows > 8192 || channels(*dims) > 2147483647LL) return GDN_ERR_UNSUPPORTED;
  if ((st = check_pool(*dims, pool)) != GDN_OK) return st;
  if ((st = check_params(params)) != GDN_OK) return st;
  if (!slot_ids || !qkv || !a || !out) return GDN_ERR_INVALID_ARG;
  DecodeArgs d = {};
  d.ssm = pool.ssm;
  d.conv = pool.conv;
  d.num_slots = pool.num_slots;
  d.conv_w = params->conv_w;
  d.conv_bias = params->conv_bias;
  d.A_log = params->A_log;
  d.dt_bias = params->dt_bias;
  d.D = params->D;
  d.slot_ids = slot_ids;
  d.B = B;
  d.qkv = qkv;
  d.a = a;
  d.out = out;
  d.err = dev_err;
  d.hk = dims->hk;
  d.hv = dims->hv;
  d.dv = dims->dv;
  d.W = dims->conv_width;
  d.C = (int32_t)channels(*dims);
  d.G = dims->hv / dims->hk;
  // Split a group's rows over 1 to 8 CTAs (at most 1024 rows each, their
  // share of shared memory): the fewest rounds of 3 CTAs per SM times a CTA's
  // rows and its prologue, which costs about as much as 128 rows of dk = 128.
  // Clusters of 8 find room for an eighth less.  64 heads of 64 in 8 groups,
  // us: 8 requests 10.8 in 4 parts (this rule), 14.0 in 8, 11.3 in 2; 16
  // requests 16.0 in 2, 19.5 in 4; 64 requests 55.9 in 2, 61.9 whole.
  const int64_t groups = (int64_t)B * d.hk, prologue = 16384 / dims->dk;
  int64_t best = INT64_MAX;
  for (int cs = 1; cs <= 8; cs *= 2) {
    const int64_t room = 3LL * sm_count() * (cs == 8 ? 7 : 8) / 8, per = (rows + cs - 1) / cs;
    const int64_t cost = (groups * cs + room - 1) / room * (per + prologue);
    if (per <= 1024 && cost <= best) {
      best = cost;
      d.cs = cs;
    }
  }
  d.rpc = (int32_t)((rows + d.cs - 1) / d.cs);
  if ((int64_t)d.hk * d.cs > 2147483647LL) return GDN_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  // The persistent form where a round of one group per SM is well filled:
  // from 0.4 of the first (64 heads of 64 in 8 groups: 4 requests, 0.21, 9.4
  // us, split 8.2; 8 requests 10.0, split 10.9), from 0.7 of the last of
  // several (24 requests, 0.63: 22.1, split 21.4; 40 requests, 0.70: 34.0,
  // split 35.0; 64 requests, 0.84: 47.9, split 56.3).
  // GDN_SSM_DECODE_PATH=ring or split (read on every call) forces one.
  const int64_t rounds = (groups + sm_count() - 1) / sm_count(), full = rounds * sm_count();
  bool ring = decode_ring_supported(*dims, B, qkv, *params) && groups * 10 >= full * (rounds == 1 ? 4 : 7);
  if (const char* path = std::getenv("GDN_SSM_DECODE_PATH")) {
    if (!std::strcmp(path, "split")) ring = false;
    if (!std::strcmp(path, "ring")) ring = decode_ring_supported(*dims, B, qkv, *params);
  }
  if (ring) {
    e = decode_ring_launch(d, dims->act_dtype, dims->conv_dtype, s);
  } else {
    switch (dims->dk) {
      case 16: e = dispatch_decode<16, 4>(d, dims->act_dtype, dims->conv_dtype, s); break;
      case 64: e = dispatch_decode<64, 8>(d, dims->act_dtype, dims->conv_dtype, s); break;
      case 128: e = dispatch_decode<128, 8>(d, dims->act_dtype, dims->conv_dtype, s); break;
    }
  }
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_SSM_DECODE);
  return GDN_OK;
}

extern "C" size_t gdn_ssm_prefill_workspace_size(const gdn_dims* dims, int32_t n_seq, int64_t total_tokens) {
  if (gdn::check_dims(dims) != GDN_OK || total_tokens <= 0 || n_seq <= 0) return 0;
  return gdn::ssm_chunk_shape(*dims) ? gdn::ssm_chunk_workspace(*dims, n_seq, total_tokens) : 0;
}

extern "C" gdn_status gdn_ssm_prefill(const gdn_dims* dims, gdn_pool pool, gdn_pool ckpt,
                                      const gdn_ssm_params* params, const int32_t* slot_ids,
                                      const int32_t* cu_seqlens, const int64_t* start_pos, int32_t n_seq,
                                      int64_t total_tokens, const int32_t* ckpt_ids, int32_t max_ckpt,
                                      int32_t ckpt_block, const void* qkv, const void* a, void* out,
                                      void* workspace, size_t workspace_bytes, uint32_t* dev_err, void* stream) {
  using namespace gdn;
  gdn_status st = check_dims(dims);
  if (st != GDN_OK) return st;
  if (n_seq < 0 || total_tokens < 0 || max_ckpt < 0) return GDN_ERR_INVALID_ARG;
  if (ckpt_block <= 0 || ckpt_block % 64) return GDN_ERR_INVALID_ARG;
  if (n_seq == 0) return GDN_OK;
  if (n_seq > 65535 || total_tokens > 2147483647LL || max_ckpt > 4 * 65535 || channels(*dims) > 2147483647LL)
    return GDN_ERR_UNSUPPORTED;
  if ((st = check_pool(*dims, pool)) != GDN_OK) return st;
  if (max_ckpt > 0 && (st = check_pool(*dims, ckpt)) != GDN_OK) return st;
  if ((st = check_params(params)) != GDN_OK) return st;
  if (!slot_ids || !cu_seqlens || !start_pos || (max_ckpt > 0 && !ckpt_ids)) return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!qkv || !a || !out)) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_ssm_prefill_workspace_size(dims, n_seq, total_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return GDN_ERR_INVALID_ARG;
  PrefillArgs p = {};
  p.ssm = pool.ssm;
  p.conv = pool.conv;
  p.num_slots = pool.num_slots;
  p.ck_ssm = ckpt.ssm;
  p.ck_num_slots = max_ckpt > 0 ? ckpt.num_slots : 0;
  p.conv_w = params->conv_w;
  p.conv_bias = params->conv_bias;
  p.A_log = params->A_log;
  p.dt_bias = params->dt_bias;
  p.D = params->D;
  p.slot_ids = slot_ids;
  p.cu_seqlens = cu_seqlens;
  p.start_pos = start_pos;
  p.n_seq = n_seq;
  p.total = total_tokens;
  p.ckpt_ids = ckpt_ids;
  p.max_ckpt = max_ckpt;
  p.ckpt_block = ckpt_block;
  p.qkv = qkv;
  p.a = a;
  p.out = out;
  p.err = dev_err;
  p.hk = dims->hk;
  p.hv = dims->hv;
  p.dk = dims->dk;
  p.dv = dims->dv;
  p.W = dims->conv_width;
  p.C = (int32_t)channels(*dims);
  p.G = dims->hv / dims->hk;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  // GDN_SSM_PREFILL_PATH=recurrent (read on every call) forces the recurrence
  const char* path = std::getenv("GDN_SSM_PREFILL_PATH");
  const bool chunked = !(path && !std::strcmp(path, "recurrent")) &&
                       ssm_chunk_supported(*dims, n_seq, total_tokens, qkv, out, *params);
  if (chunked) {
    e = ssm_chunk_launch(p, *dims, ckpt.conv, workspace, s);
  } else {
    switch (dims->dk) {
      case 16: e = dispatch_recurrent<16, 2>(p, dims->act_dtype, dims->conv_dtype, s); break;
      case 64: e = dispatch_recurrent<64, 4>(p, dims->act_dtype, dims->conv_dtype, s); break;
      case 128: e = dispatch_recurrent<128, 8>(p, dims->act_dtype, dims->conv_dtype, s); break;
    }
    if (e == cudaSuccess)
      e = conv_history_launch(*dims, pool, ckpt, slot_ids, cu_seqlens, start_pos, n_seq, total_tokens, ckpt_ids,
                              max_ckpt, ckpt_block, qkv, dev_err, s);
  }
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  count_launch(GDN_K_SSM_PREFILL);
  return GDN_OK;
}
