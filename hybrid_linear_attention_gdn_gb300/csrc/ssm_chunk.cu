// Chunked prefill of the selective state space step on the 5th-generation
// tensor cores (dk = 128, dv 64 or 128, conv width 4, bf16 activations and
// conv history).
//
// The published chunk form (Dao & Gu, "Transformers are SSMs", ICML 2024), in
// chunks of 64 tokens aligned to absolute positions.  With the cumulative log
// decay b inside the chunk and per V head
//   P_ij = (q_i . k_j) e^{b_i - b_j} dt_j   (j <= i; + D on the diagonal)
//   O    = P V + diag(e^b) Q S
//   S    <- e^{b_last} S + sum_j e^{b_last - b_j} dt_j k_j v_j^T
// q, k and q.k belong to the group, everything else to the head.  So:
//
// features kernel (chunk, group): conv1d + SiLU of the group's q and k
//   channels once instead of once per head, and G = Q K^T, written in the
//   chain kernel's operand layouts (56 KB per chunk and group, read back
//   through L2 by the heads of the group, whose chains run side by side).
// chain kernel (128 V channels = one head of 128 or two of 64; sequence or
//   segment of one): walks its chunks in order, V rows in the tensor core's
//   M = 128 rows.  Per chunk, with S^T [dv][dk] in registers between chunks:
//     O1^T = S^T Q^T         S^T the A operand in TMEM
//     O2^T = V^T P^T         V^T the A operand in TMEM; two heads' P^T side
//                            by side (N = 128), each head's rows taken from
//                            its own half
//     dS^T = (V w)^T K       w_j = e^{b_last - b_j} dt_j
//     S^T <- e^{b_last} S^T + dS^T   fp32 on the CUDA cores, rounded to
//                            nearest: the tensor core's truncating
//                            accumulation never touches the long-lived state
//   All operands are fp16 (kind::f16, four times the measured rate of
//   kind::tf32 at the same 11 bits) after exact power-of-two scalings: by the
//   largest |q| and |k| of a chunk and group, the largest |v| of a chunk and
//   head, and by upper bounds of |v w|, |P| and |S| of a head.  fp16 keeps 11
//   bits over 29 binades below the largest value or its bound (a bound may be
//   loose by 2^14), so inputs of any size do (tests from 1e-12 to 1e36), and
//   what is smaller yet than its chunk's largest loses bits.  Where the product
//   of two operands' largest magnitudes passes fp32 the result may be infinite
//   though the largest do not meet.  Roundings: the output products' operands
//   to 11 bits (at most 2^-11 of their terms, against 2^-8 of the bf16 output);
//   the state's operands to two halves each, 22 bits, in three products.
// The work per 64 x 128 V values is bound by the instructions of the
// elementwise steps (conv + SiLU, P, operand conversion), not by the products
// (tensor pipe 24 % busy) or by memory.  Measured, 64 heads of 64 in 8 groups:
// 4 x 8192 tokens 418 us (features 85, chain 333: 2.6 us per chunk; 112 us of
// memory traffic), seven ragged sequences of 3,968 tokens 141 us, 37 tokens 20
// us in a graph; 32 heads in one group, 1 x 8192 tokens 97 us (features 10,
// states of 8 segments 33, chains 54).
//
// Segments: where sequences times V tiles are too few for the SMs, each
// sequence is cut into segments of seg_chunks chunks.  A first launch walks
// all segments but each sequence's last for their state alone (K and V w: a
// third of the work), from zero (the first from the slot's state); the second
// launch starts each segment from its predecessors' states, joined in order
// with the segments' total decays, and no CTA of it reads a state that
// another may overwrite.
#include "ssm.cuh"
#include "ssm_chunk.cuh"
#include "decode_tma.cuh"  // sm_count
#include "prefill_history.cuh"
#include "tma.cuh"
#include "umma.cuh"

#include <cuda_fp16.h>

#include <cstddef>

namespace gdn {
namespace {

using namespace ssm;

constexpr int kC = 64;    // tokens per chunk
constexpr int kDK = 128;  // state size
constexpr int kRawRows = kC + 3;

// ---- workspace ----------------------------------------------------------------
// Sequence n's chunks occupy the slots from first_slot(cu[n], n) on.  A sequence
// of len tokens touches at most min(len / 64 + 2, len) chunks, and both of the
// numbers whose smaller one first_slot is grow by at least that much: the
// ranges are disjoint without a scan, and no more than one slot per token.
// Its segments likewise: from that / seg_chunks + n on.
__host__ __device__ __forceinline__ int64_t first_slot(int64_t tokens, int64_t n) {
  const int64_t by_chunk = tokens / kC + 2 * n;
  return by_chunk < tokens ? by_chunk : tokens;
}
// One record per (chunk slot, group), of fp16 operands in the tensor core's
// 128-byte swizzled layout:
struct __align__(1024) Record {
  uint8_t q[2 * 64 * 128];  // q 2^qe [token][dk], 64-column blocks of 8 KB
  uint8_t kh[128 * 128];    // k^T 2^ke [dk][token]: high halves
  uint8_t kl[128 * 128];    //   low halves
  uint8_t g[64 * 128];      // G 2^(qe + ke - 22) [i][j]
  int32_t qe, ke;
};
constexpr uint32_t kQKBytes = offsetof(Record, g), kGBytes = sizeof(Record::g), kGMBytes = kGBytes + 16;

struct ChunkArgs {
  PrefillArgs p;
  Record* rec;           // [chunk slots][hk]
  __nv_bfloat16* vhist;  // [n_seq][3][hv dv]: the V channels' conv history before the call
  float* seg_state;      // [segment slots][hv][dv][dk]
  float* seg_decay;      // [segment slots][hv]
  int32_t n_chunks, n_segs;  // slots
  int32_t seg_chunks, feat_chunks;
  int32_t hist_blocks, hist_groups;  // the history work items: sequences x channel blocks
  pfx::PrefillArgs hist;
};

struct Seq {
  int64_t t0, len, p0, p1;
  int32_t slot;
  int32_t nch;        // chunks
  int64_t first;      // first chunk slot
};
// sequence n; false: inconsistent offsets (bad = 1) or nothing to do
__device__ __forceinline__ bool load_seq(const PrefillArgs& a, int n, Seq& s, bool& bad) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  s.t0 = cu[n];
  s.len = (int64_t)cu[n + 1] - s.t0;
  s.p0 = GDN_GV(a.start_pos, a.n_seq)[n];
  s.p1 = s.p0 + s.len;
  s.slot = GDN_GV(a.slot_ids, a.n_seq)[n];
  bad = s.t0 < 0 || s.len < 0 || s.t0 + s.len > a.total || s.p0 < 0;
  if (bad) return false;
  s.nch = s.len ? (int)((s.p1 + kC - 1) / kC - s.p0 / kC) : 0;
  s.first = first_slot(s.t0, n);
  return s.len > 0;
}
// The last sequence whose first chunk slot, or segment slot (segs: chunk slot /
// div + n), is at most `slot`: one warp, 32 candidates at a time.  Offsets
// outside [0, total] end the search early, never outside the array.
__device__ __forceinline__ int find_seq(const PrefillArgs& a, int64_t slot, int div, bool segs) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n_seq;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    bool le = false;
    if (i < n) {
      const int64_t c = first_slot(cu[lo + i], lo + i);
      le = (segs ? c / div + (lo + i) : c) <= slot;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

__device__ __forceinline__ float silu_acc(float y) { return __fdividef(y, 1.f + exp_ftz(-y)); }

// The power of two 2^e that takes a largest magnitude m to [2^14, 2^15), as
// an exponent: fp16's high halves stay finite and the low halves keep 11 more
// bits of everything down to 2^-28 of m.  At most 100, which is also what a
// largest magnitude of 0 gets: operands that are all zero must not count as
// large where a bound is taken from their scales.  0 for an infinite m or NaN.
__device__ __forceinline__ int scale_exp(uint32_t m_bits) {
  const int ex = (int)(m_bits >> 23);
  if (ex == 0) return 100;
  if (ex == 255) return 0;
  const int e = 14 - (ex - 127);
  return e > 100 ? 100 : e;
}
constexpr float kLargest = 3.40282347e38f;  // of fp32
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// two values as fp16 high halves and the low halves that remain
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 r = fma2(__half22float2(h), make_float2(-1.f, -1.f), x);
  const __half2 l = __floats2half2_rn(r.x, r.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// ---------------------------------------------------------------------------
// features of q and k, G = Q K^T
// ---------------------------------------------------------------------------
// A CTA of 256 threads walks feat_chunks consecutive chunk slots of one group;
// a thread has a channel pair and half of the chunk's tokens.  67 x 512 bytes
// in, 56 KB out: 84 us for 4 x 8192 tokens of 8 groups, 0.65 of the copy
// bandwidth (issue slots 43 % busy; one chunk per CTA, its rows not requested
// ahead, took 108).  The next chunk's raw rows arrive by TMA while the
// last ones' features, already in registers, are worked on.  q and k stand
// one above the other as one 128-row operand, so that one product of M = 128
// gives G in its upper half.
constexpr int kFT = 256;
struct __align__(1024) FeatSmem {
  uint8_t qk[2 * 128 * 128];  // [q; k] [token][dk], 64-column blocks of 16 KB
  uint8_t kt[2 * 128 * 128];  // kh, kl
  uint8_t g[kGBytes];
  __align__(16) int32_t meta[4];  // qe, ke
  __align__(128) __nv_bfloat16 raw[2][kRawRows][128];  // q, k
  Seq seq;        // of the chunk whose raw rows are in raw or on their way
  int64_t chunk;  // its slot and its number in the sequence; slot -1: no more
  int32_t c;
  uint64_t raw_bar, bar;
  uint32_t qkmax[2][2], tmem_base;  // by parity; q, k
};

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(smem_addr(src)),
               "r"(bytes)
               : "memory");
}

// Sequence n, by hk CTAs of which this is number `part`: errors reported, an
// unusable slot's rows zeroed, and the V channels' conv history kept aside,
// so that the chain launch may both start chains from it and replace it.
__device__ __forceinline__ void sequence_block(const ChunkArgs& a, const int n, const int part) {
  const PrefillArgs& p = a.p;
  Seq s;
  bool bad;
  const bool some = load_seq(p, n, s, bad);
  const int cls = slot_class(s.slot, p.num_slots);
  if (part == 0 && threadIdx.x == 0) {
    if (bad) report(p.err, GDN_DEV_ERR_SEQLENS);
    else if (cls == 2) report(p.err, GDN_DEV_ERR_SLOT_OOB);
  }
  if (!some) return;
  const int64_t row = (int64_t)p.hv * p.dv / 8, step = (int64_t)p.hk * kFT;  // 16-byte pieces
  const int64_t first = (int64_t)part * kFT + threadIdx.x;
  if (cls) {
    const auto out = GDN_GV(reinterpret_cast<uint4*>(p.out), p.total * row);
    for (int64_t e = first; e < s.len * row; e += step) out[s.t0 * row + e] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const auto hist = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.conv), (long long)p.num_slots * 3 * p.C) +
                    (size_t)s.slot * 3 * p.C;
  const auto to = GDN_GV(reinterpret_cast<uint4*>(a.vhist), (long long)p.n_seq * 3 * row);
  for (int64_t e = first; e < 3 * row; e += step)
    to[(int64_t)n * 3 * row + e] = vec_at<const uint4>(hist, e / row * p.C + 2 * p.hk * kDK + e % row * 8);
}

__global__ void __launch_bounds__(kFT, 2)
    ssm_features_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  FeatSmem& S = *reinterpret_cast<FeatSmem*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const PrefillArgs& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hq = blockIdx.y;
  const int64_t slot0 = (int64_t)blockIdx.x * a.feat_chunks, slot1 = min(slot0 + a.feat_chunks, (int64_t)a.n_chunks);
  pdl_wait();
  pdl_trigger();
  if (slot0 >= a.n_chunks) {
    sequence_block(a, (int)(blockIdx.x - (a.n_chunks + a.feat_chunks - 1) / a.feat_chunks), hq);
    return;
  }
  // warp 0: the next chunk in [from, slot1) that a usable sequence has, its
  // raw rows on their way
  auto next = [&](int64_t from) {
    Seq s;
    bool bad;
    int64_t at = -1;
    int c = 0;
    for (int64_t k = from; k < slot1; ++k) {
      const int n = find_seq(p, k, 1, false);
      if (!load_seq(p, n, s, bad) || slot_class(s.slot, p.num_slots)) continue;
      if (k - s.first < 0 || k - s.first >= s.nch) continue;
      at = k;
      c = (int)(k - s.first);
      break;
    }
    if (lane == 0) {
      S.seq = s;
      S.chunk = at;
      S.c = c;
      if (at >= 0) {
        const int32_t row0 = (int32_t)(s.t0 + ((s.p0 / kC + c) * kC - 3 - s.p0));  // may be < 0: zeros
        mbar_arrive_expect_tx(&S.raw_bar, (uint32_t)sizeof(S.raw));
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (GDN_SPAN_G((hq + q * p.hk) * kDK, kDK, p.C) && GDN_SBYTES(&S.raw[q][0][0], sizeof(S.raw[0]), S))
            tma_load_2d(&S.raw[q][0][0], &xmap, (hq + q * p.hk) * kDK, row0, &S.raw_bar);
      }
    }
  };
  if (warp == 1) umma::tmem_alloc(&S.tmem_base, 64);
  if (warp == 0) {
    if (lane == 0) {
      mbar_init(&S.raw_bar, 1);
      mbar_init(&S.bar, 1);
      S.qkmax[0][0] = S.qkmax[0][1] = S.qkmax[1][0] = S.qkmax[1][1] = 0;
      fence_mbar_init();
    }
    __syncwarp();
    next(slot0);
  }
  const int cp = tid & 63;                 // channel pair of the part
  const bool isq = (tid & 64) == 0;        // warps 0, 1, 4, 5
  const int half = tid >> 7;               // tokens 32 half ..
  const int ch = (isq ? hq : p.hk + hq) * kDK + 2 * cp;
  const auto cw = GDN_GV(p.conv_w, (long long)p.C * 4);
  const float4 w0 = vec_at<const float4>(cw, (size_t)ch * 4), w1 = vec_at<const float4>(cw, (size_t)ch * 4 + 4);
  float2 bias = make_float2(0.f, 0.f);
  if (p.conv_bias) {
    const auto cb = GDN_GV(p.conv_bias, p.C);
    bias = make_float2(cb[ch], cb[ch + 1]);
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = S.tmem_base;
  bool failed = false;
  uint32_t par = 0;
#pragma unroll 1
  for (int it = 0;; ++it) {
    const int64_t cslot = S.chunk;
    if (cslot < 0) break;
    par = it & 1;
    // the first token of this thread in the sequence's tokens (may be < 0), and their number
    const int64_t m0 = (S.seq.p0 / kC + S.c) * kC + 32 * half - S.seq.p0;
    const int tlo = (int)max((int64_t)-64, -m0), thi = (int)min((int64_t)64, S.seq.len - m0);  // valid: [tlo, thi)
    const bool late = !mbar_wait(&S.raw_bar, par);
    const int64_t c0 = m0 - 32 * half;  // the chunk's first token
    if (c0 < 3) {
      // up to 3 rows before the sequence, from the history
      const auto hist = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.conv), (long long)p.num_slots * 3 * p.C) +
                        (size_t)S.seq.slot * 3 * p.C;
      for (int e = tid; e < 2 * 3 * 128; e += kFT) {
        const int q = e / (3 * 128), j = e / 128 % 3, cc = e % 128;  // history row j: token j - 3
        const int64_t r = j - c0;
        if (r >= 0 && r < kRawRows)
          S.raw[q][GDN_S((int)r, kRawRows)][cc] = hist[(size_t)j * p.C + (hq + q * p.hk) * kDK + cc];
      }
      umma::fence_proxy_async();  // before the next chunk's copy into these rows
    }
    if ((failed = __syncthreads_or(late))) break;
    float2 y[32];
    float mx = 0.f;
    {
      const auto src = GDN_SV(reinterpret_cast<const __nv_bfloat162*>(&S.raw[isq ? 0 : 1][0][0]), kRawRows * 64) +
                       (32 * half * 64 + cp);
      const float2 v0 = make_float2(w0.x, w1.x), v1 = make_float2(w0.y, w1.y), v2 = make_float2(w0.z, w1.z),
                   v3 = make_float2(w0.w, w1.w);
      float2 x0 = __bfloat1622float2(src[0]), x1 = __bfloat1622float2(src[64]), x2 = __bfloat1622float2(src[128]);
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        const float2 x3 = __bfloat1622float2(src[(t + 3) * 64]);
        float2 acc = fma2(v0, x0, bias);
        acc = fma2(v1, x1, acc);
        acc = fma2(v2, x2, acc);
        acc = fma2(v3, x3, acc);
        y[t] = make_float2(silu_acc(acc.x), silu_acc(acc.y));
        x0 = x1;
        x1 = x2;
        x2 = x3;
      }
    }
    if (tlo > 0 || thi < 32) {
#pragma unroll
      for (int t = 0; t < 32; ++t)
        if (t < tlo || t >= thi) y[t] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      const float u = fabsf(y[t].x), v = fabsf(y[t].y);  // the finite ones
      mx = fmaxf(mx, fmaxf(u <= kLargest ? u : 0.f, v <= kLargest ? v : 0.f));
    }
    {
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
      if (lane == 0) atomicMax(&S.qkmax[par][isq ? 0 : 1], m);
    }
    if (tid == 0) bulk_wait_read();  // the last chunk's record has left
    __syncthreads();  // the maxima complete, the raw rows read, the tiles free
    const int qe = scale_exp(S.qkmax[par][0]), ke = scale_exp(S.qkmax[par][1]);
    if (tid == 0) S.qkmax[par ^ 1][0] = S.qkmax[par ^ 1][1] = 0;
    {
      const float f = exp2_int(isq ? qe : ke);
      const int R0 = (isq ? 0 : kC) + 32 * half;
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        y[t] = mul2(y[t], make_float2(f, f));
        tile_at<__half2>(S.qk, sizeof(S.qk), umma::sw128_off(R0 + t, 2 * cp, 128 * 128)) =
            __floats2half2_rn(y[t].x, y[t].y);
      }
    }
    umma::fence_proxy_async();
    umma::fence_before();
    __syncthreads();  // [q; k] written
    umma::fence_after();
    const int64_t ri = cslot * p.hk + hq;
    Record& rec = a.rec[ri];
    [[maybe_unused]] const bool rec_ok = GDN_SPAN_G(ri, 1, (long long)a.n_chunks * p.hk);
    if (tid == 0) {
      const uint64_t dq = umma::desc(smem_addr(S.qk), 16, 1024);
      constexpr uint32_t ID = umma::idesc_f16(128, kC, false, false);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t ko = (k >> 2) * 16384 + (k & 3) * 32;
        umma::mma_bf16(tmem, umma::adv(dq, ko), umma::adv(dq, ko + 8192), ID, k > 0);
      }
      umma::commit(&S.bar);
      S.meta[0] = qe;
      S.meta[1] = ke;
    }
    __syncwarp();
    if (warp == 0) next(cslot + 1);
    if (!isq) {
#pragma unroll
      for (int t8 = 0; t8 < 4; ++t8) {
        uint32_t h0[4], l0[4], h1[4], l1[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = y[8 * t8 + 2 * i], v = y[8 * t8 + 2 * i + 1];
          split2(make_float2(u.x, v.x), h0[i], l0[i]);
          split2(make_float2(u.y, v.y), h1[i], l1[i]);
        }
        const uint32_t o0 = umma::sw128_off(2 * cp, 32 * half + 8 * t8, 0),
                       o1 = umma::sw128_off(2 * cp + 1, 32 * half + 8 * t8, 0);
        tile_at<uint4>(S.kt, sizeof(S.kt), o0) = make_uint4(h0[0], h0[1], h0[2], h0[3]);
        tile_at<uint4>(S.kt, sizeof(S.kt), o0 + 16384) = make_uint4(l0[0], l0[1], l0[2], l0[3]);
        tile_at<uint4>(S.kt, sizeof(S.kt), o1) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
        tile_at<uint4>(S.kt, sizeof(S.kt), o1 + 16384) = make_uint4(l1[0], l1[1], l1[2], l1[3]);
      }
    }
    if ((failed = __syncthreads_or(!mbar_wait(&S.bar, par)))) break;
    if (isq) {
      umma::fence_after();
      const int i = 32 * (warp & 3) + lane;
      float v[32];
      umma::tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 32 * half, v);
      // |v| <= 128 2^15 2^15: times 2^-22 it fits fp16
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 x = __floats2half2_rn(v[8 * q + 2 * e] * 0x1p-22f, v[8 * q + 2 * e + 1] * 0x1p-22f);
          h[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        tile_at<uint4>(S.g, sizeof(S.g), umma::sw128_off(i, 32 * half + 8 * q, 0)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
    umma::fence_proxy_async();
    umma::fence_before();
    __syncthreads();
    if (tid == 0 && rec_ok) {
      bulk_s2g(rec.q, S.qk, 8192);
      bulk_s2g(rec.q + 8192, S.qk + 16384, 8192);
      bulk_s2g(rec.kh, S.kt, 32768);  // and kl
      bulk_s2g(rec.g, S.g, kGMBytes);  // and qe, ke
      bulk_commit();
    }
  }
  if (failed && tid == 0) {
    // let what is in flight land before the memory goes
    report(p.err, GDN_DEV_ERR_TIMEOUT);
    mbar_wait(&S.raw_bar, par);
    mbar_wait(&S.raw_bar, par ^ 1);
    mbar_wait(&S.bar, par);
  }
  if (tid == 0) bulk_wait_all();
  umma::fence_before();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(tmem, 64);
}
static_assert(offsetof(FeatSmem, meta) == offsetof(FeatSmem, g) + kGBytes &&
                  offsetof(Record, qe) == offsetof(Record, g) + kGBytes,
              "G and its exponents leave and arrive as one piece");

// ---------------------------------------------------------------------------
// the chain
// ---------------------------------------------------------------------------
// Twenty-four warps, with no barrier among them after the start, only
// mbarriers:
//   0..15    compute: while the tensor core runs chunk i's products, V of chunk
//            i + 1 (kept in registers); then the state, chunk i + 1's operands
//            in place of chunk i's, and chunk i's output to its rows
//   16..19   P of chunk i + 1, the other of two buffers
//   20       issuer: every product and the copies of q and k (a thread that
//            issues products is held up about as long as they run)
//   21, 22   gates and scales of one head each
//   23       loader: the copies of raw V rows and G, the three rows before a
//            sequence from the conv history, and the largest raw input
// What bounds a chunk is instruction issue: 3,400 instructions per scheduler
// and chunk, 70 to 80 % of its slots.  It is not the products: leaving out half of
// dS^T's changed nothing.  4 x 8192 tokens: P in the compute warps cost 21 us
// more; without P at all (wrong) it would be 25 us less.
constexpr int kCompute = 512, kAux = 128;  // threads
constexpr int kIssuer = (kCompute + kAux) / 32, kLoader = kIssuer + 3;
constexpr int kThreads = 32 * (kLoader + 1);
// Registers per thread after the split of the launch's 768 x 80.  Spills cost
// more here than elsewhere: shared memory leaves little of the L1 cache (4 x
// 8192 tokens 422 us with this split, 528 with 96 / 56 / 40 and 64 bytes of the
// issuer's and the loader's spilled, 436 with 96 / 40 / 56, 450 with 88 / 64 /
// 64 and the compute warps' spilled).
constexpr int kComputeRegs = 96, kAuxRegs = 48, kHelpRegs = 48;
static_assert(kCompute * kComputeRegs + kAux * kAuxRegs + 128 * kHelpRegs <= kThreads * 80,
              "no more than the launch's registers");

// Raw V rows and G of up to kRing chunks are on their way or being read (two
// cost 6 us of 4 x 8192 tokens: copy, largest input and scales then follow one
// another within a chunk); gates in twice as many slots.
constexpr int kRing = 3, kSlots = 2 * kRing;
__device__ __forceinline__ int ring(int i) { return i % kRing; }
__device__ __forceinline__ uint32_t phase(int i) { return i / kRing & 1; }

// TMEM columns (fp16 operands hold two values per column)
constexpr uint32_t TM_DS = 0;    // dS^T [dv rows][dk]
constexpr uint32_t TM_O1 = 128;  // [dv rows][64 tokens]
constexpr uint32_t TM_O2 = 192;  // [dv rows][64 tokens of each head]
constexpr uint32_t TM_S = 320;   // S^T fp16 [dv rows][dk], 64 columns
constexpr uint32_t TM_V = 384;   // V^T fp16 [dv rows][64 tokens], 32 columns
constexpr uint32_t TM_WH = 416;  // (V w)^T fp16: high halves, 32 columns
constexpr uint32_t TM_WL = 448;  //   low halves
constexpr uint32_t TM_COLS = 512;

// Per chunk and head: e^{b_last}; with V 2^ve, (V w) 2^we, P 2^pe, q 2^qe,
// k 2^ke the operands, the factors that take the products back and forth.
struct __align__(16) Scales {
  float dec;    // e^{b_last}
  float ds;     // 2^-(we + ke)
  float o2;     // 2^-(ve + pe)
  float q;      // 2^-qe
  float grow;   // bound of what the chunk adds to |S|
  float v;      // 2^-ve
  float p;      // 2^(22 - qe - ke + pe): from the stored G to P 2^pe
  float skip;   // D 2^pe
};

// What a CTA walks: kept in shared memory, so that no role holds what another
// needs in registers.  Tokens are counted from the sequence's first.
struct Chain {
  int64_t rec0, seg0;  // record of the first chunk (and the tile's group); the sequence's first segment slot
  int32_t nit;         // chunks; 0: nothing to do
  int32_t m0;          // the first chunk's first token (-63 .. in a first segment)
  int32_t len, t0;     // tokens of the sequence; its first packed row
  int32_t n, slot, seg, n_seg;
  int32_t to_ckpt, ck_idx;  // chunks before the one that ends at the next block boundary; that boundary's index
};

template <int NH>
struct __align__(1024) ChainSmem {
  uint8_t qk[2][kQKBytes];         // q, kh, kl
  uint8_t pt[2][NH * 64 * 128];    // P 2^pe [head, i][j]
  struct __align__(1024) Gm {
    uint8_t g[kGBytes];
    int32_t meta[4];               // qe, ke
  } g[kRing];
  __nv_bfloat16 raw[kRing][kRawRows][128];
  // per chunk (mod kSlots) and head
  __align__(16) float b2[kSlots][NH][kC];  // b log2(e)
  float eb[kSlots][NH][kC];                // e^b
  float dt[kSlots][NH][kC];
  float v[kSlots][NH][kC];                 // e^{b' - b} dt, b' at the end of the token's 16-token block
  float w[kSlots][NH][kC];                 // e^{b_last - b} dt 2^(we - ve)
  Scales sc[kSlots][NH];
  float xmax[kRing][NH];              // largest raw input of a chunk, of a head
  float vgain[NH], vbias[NH];         // |V| <= vgain xmax + vbias
  uint32_t smax[NH];                  // largest |S| entering the segment, float bits
  uint64_t x_bar[kRing], g_bar[kRing], qk_bar[2];  // copies landed
  uint64_t hx[kRing];                 // xmax known, history rows in place
  uint64_t gx[kRing];                 // gates and scales known
  uint64_t used[kRing];               // raw rows and G read
  uint64_t ready;                     // operands in place
  uint64_t ds_bar, o_bar;             // dS^T done; all products done
  uint64_t s_used;                    // the state's way through S.qk is free
  uint32_t tmem_base;
  Chain ch;
};

// 8 or 16 consecutive columns of this thread's TMEM lane, written; done after
// tmem_wait_st()
__device__ __forceinline__ void tmem_put8(uint32_t taddr, const uint32_t (&v)[8], int line = __builtin_LINE()) {
  if (!umma::tmem_ok(taddr, 8, true, line)) return;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&v)[16], int line = __builtin_LINE()) {
  if (!umma::tmem_ok(taddr, 16, true, line)) return;
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// two runs of 16 columns read at once
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float (&va)[16], float (&vb)[16],
                                            int line = __builtin_LINE()) {
  if (!umma::tmem_ok(ta, 16, true, line) || !umma::tmem_ok(tb, 16, true, line)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) va[i] = vb[i] = 0.f;
    return;
  }
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%33];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(va[0]), "=f"(va[1]), "=f"(va[2]), "=f"(va[3]), "=f"(va[4]), "=f"(va[5]), "=f"(va[6]), "=f"(va[7]),
        "=f"(va[8]), "=f"(va[9]), "=f"(va[10]), "=f"(va[11]), "=f"(va[12]), "=f"(va[13]), "=f"(va[14]), "=f"(va[15]),
        "=f"(vb[0]), "=f"(vb[1]), "=f"(vb[2]), "=f"(vb[3]), "=f"(vb[4]), "=f"(vb[5]), "=f"(vb[6]), "=f"(vb[7]),
        "=f"(vb[8]), "=f"(vb[9]), "=f"(vb[10]), "=f"(vb[11]), "=f"(vb[12]), "=f"(vb[13]), "=f"(vb[14]), "=f"(vb[15])
      : "r"(ta), "r"(tb)
      : "memory");
}
// 32 bytes to a 32-byte aligned place
__device__ __forceinline__ void st_global32(float* to, float4 a, float4 b) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to), "f"(a.x), "f"(a.y), "f"(a.z), "f"(a.w),
               "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
               : "memory");
}
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// D (TMEM) (+)= A B with A in TMEM (fp16 pairs: K = 16 is 8 columns from
// tmem_a) and B from a shared-memory descriptor, kind::f16
__device__ __forceinline__ void mma_f16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc,
                                           bool accumulate, int line = __builtin_LINE()) {
  if (!umma::tmem_ok(tmem_d, umma::idesc_n(idesc), false, line) || !umma::tmem_ok(tmem_a, 8, false, line)) return;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// grid (V tiles, segment slots); NH heads of 128 / NH channels per tile.
// STATE: the segment's state alone (every segment but a sequence's last).
template <int NH, bool STATE>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_chain_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap xmap) {
  constexpr int DV = 128 / NH;
  constexpr int kPart = (kCompute + (STATE ? 0 : kAux)) / 32;  // warps that take part in a chunk
  using SM = ChainSmem<NH>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  SM& S = *reinterpret_cast<SM*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const PrefillArgs& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x, h0 = tile * NH, hq = h0 / p.G;
  pdl_wait();
  pdl_trigger();
  if (!STATE && (int)blockIdx.y >= a.n_segs) {
    // the conv histories of checkpoints and final states: after the chains,
    // on the SMs that they leave free
    const int item = ((int)blockIdx.y - a.n_segs) * (int)gridDim.x + (int)blockIdx.x;
    if (item < p.n_seq * a.hist_blocks)
      for (int grp = 0; grp < a.hist_groups; ++grp)
        pfx::history_channel<__nv_bfloat16, __nv_bfloat16>(a.hist, item / a.hist_blocks, grp,
                                                           item % a.hist_blocks * kThreads + tid);
    return;
  }
  if (warp == 0) {
    // inconsistent, empty and padded sequences are the features kernel's
    const int n = find_seq(p, blockIdx.y, a.seg_chunks, true);
    Seq s;
    bool bad;
    Chain c = {};
    if (load_seq(p, n, s, bad) && !slot_class(s.slot, p.num_slots)) {
      c.seg0 = s.first / a.seg_chunks + n;
      c.seg = (int)(blockIdx.y - c.seg0);
      c.n_seg = (s.nch + a.seg_chunks - 1) / a.seg_chunks;
      if (c.seg >= 0 && c.seg < c.n_seg && !(STATE && c.seg == c.n_seg - 1)) {
        const int first = c.seg * a.seg_chunks;  // chunk of the sequence
        const int64_t P = s.p0 / kC + first;     // and absolute
        const int kpc = p.ckpt_block / kC;
        c.nit = min(s.nch - first, a.seg_chunks);
        c.rec0 = (s.first + first) * p.hk + hq;
        c.m0 = first * kC - (int)(s.p0 % kC);
        c.len = (int)s.len;
        c.t0 = (int)s.t0;
        c.n = n;
        c.slot = s.slot;
        c.to_ckpt = kpc - 1 - (int)(P % kpc);
        c.ck_idx = (int)min((int64_t)p.max_ckpt, P / kpc - s.p0 / p.ckpt_block);
      }
    }
    if (lane == 0) S.ch = c;
  } else if (warp == 1) {
    umma::tmem_alloc(&S.tmem_base, TM_COLS);
  } else if (tid == 64) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&S.x_bar[i], 1);
      mbar_init(&S.g_bar[i], 1);
      mbar_init(&S.hx[i], 1);
      mbar_init(&S.gx[i], NH);
      mbar_init(&S.used[i], kPart);
    }
    mbar_init(&S.qk_bar[0], 1);
    mbar_init(&S.qk_bar[1], 1);
    mbar_init(&S.ready, kPart);
    mbar_init(&S.ds_bar, 1);
    mbar_init(&S.o_bar, 1);
    mbar_init(&S.s_used, kCompute / 32);
#pragma unroll
    for (int i = 0; i < NH; ++i) S.smax[i] = 0;
    fence_mbar_init();
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const int nit = S.ch.nit;
  if (nit == 0) {
    if (warp == 1) umma::tmem_dealloc(S.tmem_base, TM_COLS);
    return;
  }
  const uint32_t tmem = S.tmem_base;
  static_assert(TM_O1 == TM_DS + kDK && TM_O2 == TM_O1 + kC && TM_S == TM_O2 + 2 * kC && TM_V == TM_S + kDK / 2 &&
                    TM_WH == TM_V + kC / 2 && TM_WL == TM_WH + kC / 2 && TM_WL + kC / 2 <= TM_COLS,
                "TMEM regions");

  auto bulk = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, bytes);
    if (GDN_GBYTES(src, bytes, a.rec, (long long)a.n_chunks * p.hk * sizeof(Record)) && GDN_SBYTES(dst, bytes, S))
      bulk_g2s(dst, src, bytes, bar);
  };
  if (warp >= kIssuer) {
    // ------------------------------------------------------------------ issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kHelpRegs));
    if (warp == kIssuer) {
      constexpr uint32_t ID_O1 = umma::idesc_f16(128, kC, false, false);
      constexpr uint32_t ID_O2 = umma::idesc_f16(128, NH * kC, false, false);
      constexpr uint32_t ID_S = umma::idesc_f16(128, kDK, false, false);
      // q and k (the state alone needs only k)
      constexpr uint32_t kSkip = STATE ? sizeof(Record::q) : 0;
      auto load_qk = [&](int i) {
        bulk(S.qk[i & 1] + kSkip, a.rec[S.ch.rec0 + (int64_t)i * p.hk].q + kSkip, kQKBytes - kSkip, &S.qk_bar[i & 1]);
      };
      int n_qk = 0, n_mma = 0;  // issued
      bool ok = __all_sync(0xffffffffu, mbar_wait(&S.s_used, 0));
      if (ok && lane == 0) {
        for (; n_qk < 2 && n_qk < nit; ++n_qk) load_qk(n_qk);
      }
      // pass i: chunk i's operands are in place
      for (int i = 0; i < nit && ok; ++i) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&S.ready, i & 1)))) break;
        if (lane == 0 && (ok = mbar_wait(&S.qk_bar[i & 1], (i >> 1) & 1))) {
          umma::fence_after();
          const uint64_t dq = umma::desc(smem_addr(S.qk[i & 1]), 16, 1024);
          const uint64_t dh = umma::adv(dq, offsetof(Record, kh)), dl = umma::adv(dq, offsetof(Record, kl));
          // dS^T = (V w)^T K, small products first; on it the next state waits
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ta(tmem + TM_DS, tmem + TM_WL + 8 * k, umma::adv(dh, 32 * k), ID_S, k > 0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ta(tmem + TM_DS, tmem + TM_WH + 8 * k, umma::adv(dl, 32 * k), ID_S, true);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ta(tmem + TM_DS, tmem + TM_WH + 8 * k, umma::adv(dh, 32 * k), ID_S, true);
          umma::commit(&S.ds_bar);
          if (!STATE) {
            // O1^T = S^T Q^T, O2^T = V^T P^T
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16_ta(tmem + TM_O1, tmem + TM_S + 8 * k, umma::adv(dq, (k >> 2) * 8192 + (k & 3) * 32), ID_O1,
                         k > 0);
            const uint64_t dp = umma::desc(smem_addr(S.pt[i & 1]), 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_ta(tmem + TM_O2, tmem + TM_V + 8 * k, umma::adv(dp, 32 * k), ID_O2, k > 0);
          }
          umma::commit(&S.o_bar);
          ++n_mma;
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (lane == 0 && ok && (ok = mbar_wait(&S.o_bar, i & 1)) && i + 2 < nit) {
          load_qk(i + 2);
          n_qk = i + 3;
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (lane == 0) {
        if (!ok) report(p.err, GDN_DEV_ERR_TIMEOUT);
        // what is in flight lands before the memory goes (at once, unless a wait expired)
        for (int k = max(0, n_qk - 2); k < n_qk; ++k) mbar_wait(&S.qk_bar[k & 1], (k >> 1) & 1);
        if (n_mma) mbar_wait(&S.o_bar, (n_mma - 1) & 1);
      }
    } else if (warp <= kIssuer + NH) {
      // ----------------------------------------------------------------- gates
      // two tokens per lane, their logits loaded one chunk ahead
      const int hh = warp - kIssuer - 1, gh = h0 + hh;
      const auto gate_a = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.a), p.total * p.hv);
      const int m0 = S.ch.m0, len = S.ch.len;
      auto gate_load = [&](int i, float (&ga)[2]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = m0 + i * kC + 32 * e + lane;
          ga[e] = i < nit && (unsigned)m < (unsigned)len
                      ? __bfloat162float(gate_a[(long long)(S.ch.t0 + m) * p.hv + gh])
                      : 0.f;
        }
      };
      const float A_log = GDN_GV(p.A_log, p.hv)[gh], dtb = GDN_GV(p.dt_bias, p.hv)[gh];
      const float D = p.D ? GDN_GV(p.D, p.hv)[gh] : 0.f;
      float ga[2];
      gate_load(0, ga);
      bool ok = true;
      for (int i = 0; i < nit && ok; ++i) {
        float dt[2], b[2], suf[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = (unsigned)(m0 + i * kC + 32 * e + lane) < (unsigned)len;
          const Gate t = gate(A_log, dtb, ga[e]);
          dt[e] = in ? t.dt : 0.f;
          b[e] = suf[e] = in ? floor_log_decay(t.g) : 0.f;
        }
        gate_load(i + 1, ga);
        // sums from the front and from the back: b_last - b_j is a sum of its
        // own, exact to its own size whatever b_last is
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float u = __shfl_up_sync(0xffffffffu, b[e], o), v = __shfl_down_sync(0xffffffffu, suf[e], o);
            if (lane >= o) b[e] += u;
            if (lane + o < 32) suf[e] += v;
          }
        }
        b[1] += __shfl_sync(0xffffffffu, b[0], 31);
        const float back = __shfl_sync(0xffffffffu, suf[1], 0), all = back + __shfl_sync(0xffffffffu, suf[0], 0);
        const float nx = __shfl_down_sync(0xffffffffu, suf[0], 1), ny = __shfl_down_sync(0xffffffffu, suf[1], 1);
        suf[0] = (lane < 31 ? nx : 0.f) + back;
        suf[1] = lane < 31 ? ny : 0.f;
        float vj[2], wj[2], eb[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          wj[e] = expf(suf[e]) * dt[e];
          eb[e] = expf(b[e]);
          b[e] *= 1.4426950408889634f;
          vj[e] = ex2(__shfl_sync(0xffffffffu, b[e], lane | 15) - b[e]) * dt[e];
        }
        // the largest finite dt and weight (a weight only decays from its dt:
        // where the decay is strong, the state holds what the last tokens
        // gave, however small beside the largest dt)
        auto largest = [](float x, float y) {
          const float m = fmaxf(x <= kLargest ? x : 0.f, y <= kLargest ? y : 0.f);
          return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        };
        const float dtm = largest(dt[0], dt[1]), wm = largest(wj[0], wj[1]);
        // Chunk i's raw rows and G have landed: chunk i - 3's were read by
        // every compute warp, whose chunk i - 5 was done before that, so the
        // slot of chunk i - 6 may be written.
        const bool in_time = mbar_wait(&S.hx[ring(i)], phase(i)) && mbar_wait(&S.g_bar[ring(i)], phase(i));
        if (!(ok = __all_sync(0xffffffffu, in_time))) break;
        const int buf = i % kSlots, qe = S.g[ring(i)].meta[0], ke = S.g[ring(i)].meta[1];
        // |V| <= vb, |V w| <= vb max w,
        // |P| <= 128 max|q| max|k| max dt + |D| < 2^(37 - qe - ke) max dt + |D|,
        // each of the two below 2^(14 - pe).  A bound that passes the largest
        // fp32 value is that value: what is finite is no larger.
        const float vb = fminf(fmaf(S.vgain[hh], S.xmax[ring(i)][hh], S.vbias[hh]), kLargest);
        const float wb = fminf(vb * wm, kLargest);
        const int ve = scale_exp(__float_as_uint(vb));
        const int we = max(ve - 126, min(ve + 126, scale_exp(__float_as_uint(wb))));
        const int pe =
            max(-126, min(scale_exp(__float_as_uint(dtm)) - (37 - qe - ke), scale_exp(__float_as_uint(fabsf(D)))) - 1);
        const float fw = exp2_int(we - ve);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 32 * e + lane;
          S.b2[buf][hh][t] = b[e];
          S.v[buf][hh][t] = vj[e];
          S.eb[buf][hh][t] = eb[e];
          S.dt[buf][hh][t] = dt[e];
          S.w[buf][hh][t] = wj[e] * fw;
        }
        if (lane == 0) {
          Scales& c = S.sc[buf][hh];
          c.dec = expf(all);
          c.ds = exp2_int(-we) * exp2_int(-ke);
          c.o2 = exp2_int(-ve) * exp2_int(-pe);
          c.q = exp2_int(-qe);
          // 64 max|V w| max|k|, in two steps: neither factor overflows alone
          c.grow = wb * exp2_int((21 - ke) / 2) * exp2_int(21 - ke - (21 - ke) / 2);
          c.v = exp2_int(-ve);
          c.p = exp2_int(max(-126, min(127, 22 - qe - ke + pe)));
          c.skip = D * exp2_int(pe);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.gx[ring(i)]);
      }
      if (!ok && lane == 0) report(p.err, GDN_DEV_ERR_TIMEOUT);
    } else if (warp == kLoader) {
      // ---------------------------------------------------------------- loader
      auto load_xg = [&](int i) {
        const int32_t row0 = S.ch.t0 + S.ch.m0 + i * kC - 3;  // may be < 0: zeros
        mbar_arrive_expect_tx(&S.x_bar[ring(i)], (uint32_t)sizeof(S.raw[0]));
        if (GDN_SPAN_G(2 * p.hk * kDK + tile * 128, 128, p.C) && GDN_SBYTES(&S.raw[ring(i)][0][0], sizeof(S.raw[0]), S))
          tma_load_2d(&S.raw[ring(i)][0][0], &xmap, 2 * p.hk * kDK + tile * 128, row0, &S.x_bar[ring(i)]);
        bulk(&S.g[ring(i)], a.rec[S.ch.rec0 + (int64_t)i * p.hk].g, kGMBytes, &S.g_bar[ring(i)]);
      };
      int n = 0;  // issued
      if (lane == 0)
        for (; n < kRing && n < nit; ++n) load_xg(n);
      n = min(kRing, nit);
      // the up to 3 rows just before the sequence, from the conv history
      __nv_bfloat16 hrow[3][4];
      if (S.ch.m0 < 3) {
        const int64_t row = (int64_t)p.hv * DV;
        const auto hist =
            GDN_GV((const __nv_bfloat16*)a.vhist, (long long)p.n_seq * 3 * row) + (size_t)S.ch.n * 3 * row;
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) hrow[j][k] = hist[j * row + tile * 128 + 32 * k + lane];
      }
      {
        // |V| <= |conv| <= max over a head's channels of sum |w| times the
        // largest raw input, plus the largest |bias|
        const auto cw = GDN_GV(p.conv_w, (long long)p.C * 4);
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          float gain = 0.f, bmax = 0.f;
#pragma unroll
          for (int k = hh * (DV / 32); k < (hh + 1) * (DV / 32); ++k) {
            const int ch = 2 * p.hk * kDK + tile * 128 + 32 * k + lane;
            const float4 w = vec_at<const float4>(cw, (size_t)ch * 4);
            gain = fmaxf(gain, fabsf(w.x) + fabsf(w.y) + fabsf(w.z) + fabsf(w.w));
            if (p.conv_bias) bmax = fmaxf(bmax, fabsf(GDN_GV(p.conv_bias, p.C)[ch]));
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            gain = fmaxf(gain, __shfl_xor_sync(0xffffffffu, gain, o));
            bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, o));
          }
          if (lane == 0) {
            S.vgain[hh] = gain;
            S.vbias[hh] = bmax;
          }
        }
      }
      bool ok = true;
      for (int i = 0; i < nit && ok; ++i) {
        // the next chunk's copies go out before this one's rows are looked at
        // (in one pass, a copy and the maximum one after the other took as
        // long as a chunk and cost 23 us of 4 x 8192 tokens)
        if (i + 1 >= kRing && i + 1 < nit) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&S.used[ring(i + 1)], phase(i + 1 - kRing))))) break;
          if (lane == 0) load_xg(i + 1);
          n = i + 2;
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&S.x_bar[ring(i)], phase(i))))) break;
        const int m0 = S.ch.m0 + i * kC;
        const auto rows = GDN_SV(reinterpret_cast<uint4*>(&S.raw[ring(i)][0][0]), kRawRows * 16);
        if (m0 < 3 || S.ch.len - m0 < kC) {
          // What stands around the sequence in the packed rows is not its
          // business: zeros, or it would count among the largest inputs.
          for (int e = lane; e < kRawRows * 16; e += 32)
            if ((unsigned)(m0 + e / 16) >= (unsigned)S.ch.len + 3) rows[e] = make_uint4(0u, 0u, 0u, 0u);
          __syncwarp();
          // history row j is token j - 3, raw row r token m0 - 3 + r
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const int r = j - m0;
            if (r >= 0 && r < kRawRows)
#pragma unroll
              for (int k = 0; k < 4; ++k) S.raw[ring(i)][GDN_S(r, kRawRows)][32 * k + lane] = hrow[j][k];
          }
          umma::fence_proxy_async();  // before a later chunk's copy into these rows
          __syncwarp();
        }
        // the largest finite |raw input| of each head: its channels are those
        // of the lanes whose 16-byte pieces (lane mod 16) are its own
        __nv_bfloat162 mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 8
        for (int e = lane; e < kRawRows * 16; e += 32) {
          const uint4 u = rows[e];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t v = w[k] & 0x7fff7fffu;
            mx[k] = __hmax2(mx[k], *reinterpret_cast<const __nv_bfloat162*>(&v));  // a NaN is passed over
          }
        }
        const float2 m01 = __bfloat1622float2(__hmax2(__hmax2(mx[0], mx[1]), __hmax2(mx[2], mx[3])));
        uint32_t m = __float_as_uint(fmaxf(m01.x, m01.y));
        if (__any_sync(0xffffffffu, m >= 0x7f800000u)) {  // infinities: without them
          m = 0;
          for (int e = lane; e < kRawRows * 16; e += 32)
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const float x = __bfloat162float(S.raw[ring(i)][e / 16][e % 16 * 8 + k]);
              const uint32_t v = __float_as_uint(x) & 0x7fffffffu;
              m = max(m, v < 0x7f800000u ? v : 0u);
            }
        }
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          const uint32_t mh = __reduce_max_sync(0xffffffffu, NH == 1 || (lane >> 3 & 1) == hh ? m : 0u);
          if (lane == 0) S.xmax[ring(i)][hh] = __uint_as_float(mh);
        }
        if (lane == 0) mbar_arrive(&S.hx[ring(i)]);
        __syncwarp();
      }
      if (lane == 0) {
        if (!ok) report(p.err, GDN_DEV_ERR_TIMEOUT);
        for (int k = max(0, n - kRing); k < n; ++k) {  // as the issuer
          mbar_wait(&S.x_bar[ring(k)], phase(k));
          mbar_wait(&S.g_bar[ring(k)], phase(k));
        }
      }
    }
  } else if (warp >= kCompute / 32) {
    // --------------------------------------------------------------------- aux
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kAuxRegs));
    if constexpr (!STATE) {
      // thread: row pr of the heads' 64 NH, in every 16-token block the PC
      // columns from pc0; what lies above the diagonal stays zero
      const int row = tid - kCompute;
      constexpr int PC = 8 * NH;
      const int pr = NH == 2 ? row : (row & 63), pi = pr & 63, ph = pr >> 6;
      const int pc0 = NH == 2 ? 0 : 8 * (row >> 6);
      const int wlo = pi & 32;  // the warp's rows: wlo .. wlo + 31 of a head
#pragma unroll
      for (int k = 0; k < 4 * PC / 8; ++k) {
        const uint32_t at = umma::sw128_off(pr, 16 * (k % 4) + pc0 + 8 * (k / 4), 0);
        tile_at<uint4>(S.pt[0], sizeof(S.pt[0]), at) = make_uint4(0u, 0u, 0u, 0u);
        tile_at<uint4>(S.pt[1], sizeof(S.pt[1]), at) = make_uint4(0u, 0u, 0u, 0u);
      }
      // P of the segment's chunk i; false (for the whole warp) if a wait expired
      auto put_p = [&](int i) -> bool {
        const uint32_t par = phase(i);
        if (!__all_sync(0xffffffffu, mbar_wait(&S.gx[ring(i)], par) && mbar_wait(&S.g_bar[ring(i)], par))) return false;
        const int buf = i % kSlots;
#pragma unroll 1
        for (int J = 0; 16 * J < wlo + 32; ++J) {
          const int pc = 16 * J + pc0;
          // P_ij = G_ij u_i v_j: both factors taken at the end b' of j's
          // 16-token block, u_i = e^{b_i - b'} at most 1 below the diagonal
          // blocks; on them it is large where the block decays, and beyond
          // 2^80 the differences are taken one by one
          const float bi = S.b2[buf][ph][pi], be = S.b2[buf][ph][GDN_S(pc | 15, kC)];
          const float pscale = S.sc[buf][ph].p;
          const float u = ex2(bi - be) * pscale;
          float2 e[PC / 2];
#pragma unroll
          for (int c8 = 0; c8 < PC / 8; ++c8) {
            const uint4 g4 = tile_at<uint4>(S.g[ring(i)].g, kGBytes, umma::sw128_off(pi, pc + 8 * c8, 0));
            const float4 va = *reinterpret_cast<const float4*>(&S.v[buf][ph][GDN_S(pc + 8 * c8, kC - 7)]);
            const float4 vb = *reinterpret_cast<const float4*>(&S.v[buf][ph][pc + 8 * c8 + 4]);
            const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
            const float2 vv[4] = {lo2(va), hi2(va), lo2(vb), hi2(vb)};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              e[4 * c8 + k] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&gw[k])),
                                   mul2(vv[k], make_float2(u, u)));
          }
          if (16 * J >= wlo) {  // the warp holds a diagonal block
            const float sk = S.sc[buf][ph].skip;
            if (__any_sync(0xffffffffu, S.b2[buf][ph][pc & ~15] - be > 80.f)) {
#pragma unroll 1
              for (int k = 0; k < PC; ++k) {
                const int j = pc + k;
                const float g = __half2float(tile_at<__half>(S.g[ring(i)].g, kGBytes, umma::sw128_off(pi, j, 0)));
                const float x = j > pi ? 0.f : g * (ex2(bi - S.b2[buf][ph][GDN_S(j, kC)]) * S.dt[buf][ph][j] * pscale);
#pragma unroll
                for (int q = 0; q < PC / 2; ++q) {
                  if (2 * q == k) e[q].x = x;
                  if (2 * q + 1 == k) e[q].y = x;
                }
              }
            }
            const int dj = pi - pc;  // the diagonal's column
#pragma unroll
            for (int k = 0; k < PC / 2; ++k) {
              e[k].x = 2 * k < dj ? e[k].x : 2 * k == dj ? e[k].x + sk : 0.f;
              e[k].y = 2 * k + 1 < dj ? e[k].y : 2 * k + 1 == dj ? e[k].y + sk : 0.f;
            }
          }
#pragma unroll
          for (int c8 = 0; c8 < PC / 8; ++c8)
            tile_at<uint4>(S.pt[i & 1], sizeof(S.pt[0]), umma::sw128_off(pr, pc + 8 * c8, 0)) =
                make_uint4(half2_bits(e[4 * c8].x, e[4 * c8].y), half2_bits(e[4 * c8 + 1].x, e[4 * c8 + 1].y),
                           half2_bits(e[4 * c8 + 2].x, e[4 * c8 + 2].y), half2_bits(e[4 * c8 + 3].x, e[4 * c8 + 3].y));
        }
        umma::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.used[ring(i)]);
        return true;
      };
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < nit; ++i) {
        // the products of chunk i - 1 are done before the next pass writes the
        // buffer that they read
        if (!(ok = __all_sync(0xffffffffu, put_p(i) && (i == 0 || mbar_wait(&S.o_bar, (i - 1) & 1))))) break;
        if (lane == 0) mbar_arrive(&S.ready);
      }
      if (!ok && lane == 0) report(p.err, GDN_DEV_ERR_TIMEOUT);
    }
  } else {
    // ----------------------------------------------------------------- compute
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kComputeRegs));
    const int lrow = 32 * (warp & 3) + lane;  // V channel of the tile, TMEM lane
    const int qq = warp >> 2;                 // token (or dk column) quarter
    const int hl = lrow / DV;                 // this row's head within the tile
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int ch = 2 * p.hk * kDK + tile * 128 + lrow;

    // the state entering the segment, S^T row lrow, columns 32 qq ..
    float2 st[16];
    float seg_dec = 1.f;
    const long long slot_n = (long long)p.hv * DV * kDK;  // a slot's state, [hv][dv][dk]
    const auto segs = GDN_GV(a.seg_state, a.n_segs * slot_n);
    // A state tile goes to and from global memory in whole rows (one per
    // warp-wide access of 16-byte pieces) and through S.qk, which is free
    // before the first chunk's operands arrive and after the last product, to
    // the threads' quarter rows: piece p of row r at p ^ (r & 7).  (Quarter
    // rows straight from global memory took 4,000 cycles a tile: 32 lines per
    // access.)
    constexpr unsigned kTile = 128 * kDK * 4;
    static_assert(kTile <= sizeof(S.qk), "the state tile's way through shared memory");
    uint8_t* const tile_smem = &S.qk[0][0];
    const size_t tile0 = (size_t)tile * 128 * kDK;
    auto piece_off = [](int r, int p) { return (uint32_t)r * 512u + (uint32_t)((p ^ (r & 7)) << 4); };
    auto save = [&](const auto& to) {  // the state to `to` (the tile's place), all compute warps
#pragma unroll
      for (int e = 0; e < 8; ++e)
        tile_at<float4>(tile_smem, kTile, piece_off(lrow, 8 * qq + e)) = join4(st[2 * e], st[2 * e + 1]);
      named_sync(1, kCompute);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        vec_at<float4>(to, ((warp + 16 * j) * 32 + lane) * 4) =
            tile_at<float4>(tile_smem, kTile, piece_off(warp + 16 * j, lane));
    };
    {
      // One segment: from the slot.  Several: the first launch starts the
      // first segment from the slot and keeps a copy, at the last segment's
      // otherwise unused place, for the second launch; the others from zero.
      const auto slot = GDN_GV(p.ssm, p.num_slots * slot_n) + ((size_t)S.ch.slot * slot_n + tile0);
      const int seg = S.ch.seg, n_seg = S.ch.n_seg;
      const int64_t seg0 = S.ch.seg0;
      const auto keep = segs + (n_seg > 1 ? (seg0 + n_seg - 1) * slot_n + (int64_t)tile0 : 0);
      float4 v[8];  // piece `lane` of rows warp, warp + 16, ..
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = ((warp + 16 * j) * 32 + lane) * 4;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (seg == 0) v[j] = STATE || n_seg == 1 ? vec_at<const float4>(slot, at) : vec_at<const float4>(keep, at);
        if (STATE && seg == 0) vec_at<float4>(keep, at) = v[j];
      }
      if (!STATE) {
        for (int k = 0; k < seg; ++k) {
          const auto L = segs + ((seg0 + k) * slot_n + (int64_t)tile0);
          const auto dec = GDN_GV(a.seg_decay, (long long)a.n_segs * p.hv) + ((seg0 + k) * p.hv + h0);
          // the first segment's state holds the slot's already
          const float d0 = k ? dec[0] : 0.f, d1 = k ? dec[NH - 1] : 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 x = vec_at<const float4>(L, ((warp + 16 * j) * 32 + lane) * 4);
            const float d = j < 4 ? d0 : d1;  // rows 64 .. are the second of two heads
            v[j].x = fmaf(d, v[j].x, x.x);
            v[j].y = fmaf(d, v[j].y, x.y);
            v[j].z = fmaf(d, v[j].z, x.z);
            v[j].w = fmaf(d, v[j].w, x.w);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) tile_at<float4>(tile_smem, kTile, piece_off(warp + 16 * j, lane)) = v[j];
      named_sync(1, kCompute);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 x = tile_at<float4>(tile_smem, kTile, piece_off(lrow, 8 * qq + e));
        st[2 * e] = lo2(x);
        st[2 * e + 1] = hi2(x);
      }
      umma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.s_used);
    }
    if (!STATE) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(st[i].x) & 0x7fffffffu, v = __float_as_uint(st[i].y) & 0x7fffffffu;
        m = max(m, max(u < 0x7f800000u ? u : 0u, v < 0x7f800000u ? v : 0u));  // the finite ones
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) atomicMax(&S.smax[hl], m);  // a warp's rows are of one head
    }
    const float4 w4 = vec_at<const float4>(GDN_GV(p.conv_w, (long long)p.C * 4), (size_t)ch * 4);
    const float bias = p.conv_bias ? GDN_GV(p.conv_bias, p.C)[ch] : 0.f;
    // chunks until the next block boundary, and the boundary's index
    int next_ckpt = S.ch.to_ckpt;  // the chunk that ends at the next block boundary
    // the sequence's tokens among the 16 from token `at` of the segment's chunks on: [lo, hi)
    auto inside = [&](int at, int& lo, int& hi) {
      lo = -S.ch.m0 - at;
      hi = min(S.ch.nit * kC, S.ch.len - S.ch.m0) - at;
    };

    float2 y[8];  // V 2^ve of the next chunk: channel lrow, tokens 16 qq ..
    // V of the segment's chunk i; false (for the whole warp) if a wait expired
    auto features = [&](int i) -> bool {
      const uint32_t par = phase(i);
      if (!__all_sync(0xffffffffu, mbar_wait(&S.gx[ring(i)], par) && mbar_wait(&S.x_bar[ring(i)], par))) return false;
      const int buf = i % kSlots;
      {
        const auto xs = GDN_SV(reinterpret_cast<const uint16_t*>(&S.raw[ring(i)][0][0]), kRawRows * 128) +
                        (16 * qq * 128 + lrow);
        uint32_t x[19];
#pragma unroll
        for (int r = 0; r < 19; ++r) x[r] = xs[r * 128];
        auto pair = [&](int r) {  // rows r, r + 1 in fp32
          return make_float2(__uint_as_float(x[r] << 16), __uint_as_float(x[r + 1] << 16));
        };
        // SiLU(v) 2^ve = v / (2^-ve + 2^-ve e^-v)
        const float cv = S.sc[buf][hl].v;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          float2 v = fma2(make_float2(w4.x, w4.x), pair(2 * t), make_float2(bias, bias));
          v = fma2(make_float2(w4.y, w4.y), pair(2 * t + 1), v);
          v = fma2(make_float2(w4.z, w4.z), pair(2 * t + 2), v);
          v = fma2(make_float2(w4.w, w4.w), pair(2 * t + 3), v);
          const float2 e = mul2(v, make_float2(-1.4426950408889634f, -1.4426950408889634f));
          const float2 d = fma2(make_float2(ex2(e.x), ex2(e.y)), make_float2(cv, cv), make_float2(cv, cv));
          y[t] = make_float2(__fdividef(v.x, d.x), __fdividef(v.y, d.y));
        }
      }
      int tlo, thi;
      inside(i * kC + 16 * qq, tlo, thi);
      if (tlo > 0 || thi < 16) {  // tokens outside the sequence
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (2 * t < tlo || 2 * t >= thi) y[t].x = 0.f;
          if (2 * t + 1 < tlo || 2 * t + 1 >= thi) y[t].y = 0.f;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.used[ring(i)]);
      return true;
    };
    // chunk i's V and V w to their operands
    auto put_v = [&](int i) {
      const auto ws = GDN_SV(&S.w[i % kSlots][hl][0], kC);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int t4 = 0; t4 < 4; ++t4) {
        const float4 w = vec_at<const float4>(ws, 16 * qq + 4 * t4);
        split2(mul2(y[2 * t4], lo2(w)), hi[2 * t4], lo[2 * t4]);
        split2(mul2(y[2 * t4 + 1], hi2(w)), hi[2 * t4 + 1], lo[2 * t4 + 1]);
      }
      tmem_put8(tlane + TM_WH + 8 * qq, hi);
      tmem_put8(tlane + TM_WL + 8 * qq, lo);
      if (!STATE) {
        uint32_t v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = half2_bits(y[t].x, y[t].y);
        tmem_put8(tlane + TM_V + 8 * qq, v);
      }
    };
    float s_bound = 0.f, s_back = 0.f;  // >= |S|; 2^-e of the S^T operand
    auto put_s = [&]() {
      if constexpr (!STATE) {
        const int se = scale_exp(__float_as_uint(s_bound));
        const float fs = exp2_int(se);
        s_back = exp2_int(-se);
        uint32_t r[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = mul2(st[e], make_float2(fs, fs));
          r[e] = half2_bits(x.x, x.y);
        }
        tmem_put16(tlane + TM_S + 16 * qq, r);
      }
    };
    auto publish = [&](uint64_t* bar) {
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };

    const auto out = GDN_GV(reinterpret_cast<__nv_bfloat16*>(p.out), p.total * p.hv * DV);
    named_sync(1, kCompute);  // smax complete
    s_bound = __uint_as_float(S.smax[hl]);
    bool ok = true;
    if ((ok = __all_sync(0xffffffffu, features(0)))) {
      put_v(0);
      put_s();
      tmem_wait_st();
      publish(&S.ready);
    }
    // pass i: chunk i + 1's V, the state after chunk i, chunk i + 1's operands
#pragma unroll 1
    for (int i = 0; i < nit && ok; ++i) {
      const bool more = i + 1 < nit;
      if (more && !(ok = __all_sync(0xffffffffu, features(i + 1)))) break;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&S.ds_bar, i & 1)))) break;
      umma::fence_after();
      const Scales& sc = S.sc[i % kSlots][hl];
      const float4 sa = *reinterpret_cast<const float4*>(&sc.dec);  // dec, ds, o2, q
      [[maybe_unused]] const float f1 = s_back * sa.w, f2 = sa.z;
      s_bound = fminf(fmaf(s_bound, sa.x, sc.grow), kLargest);
      seg_dec *= sa.x;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float d[16];
        umma::tmem_ld16(tlane + TM_DS + 32 * qq + 16 * k, d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          st[8 * k + e] = fma2(st[8 * k + e], make_float2(sa.x, sa.x),
                               mul2(make_float2(d[2 * e], d[2 * e + 1]), make_float2(sa.y, sa.y)));
      }
      // the products of chunk i are done: their operands may go
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&S.o_bar, i & 1)))) break;
      umma::fence_after();
      if (more) {
        put_v(i + 1);
        put_s();
      }
      [[maybe_unused]] float o1[16], o2[16];
      if (!STATE)
        tmem_ld16x2(tlane + TM_O1 + 16 * qq, tlane + TM_O2 + (NH == 2 ? hl * kC : 0) + 16 * qq, o1, o2);
      if (more) {
        tmem_wait_st();
        publish(&S.ready);
      }
      if constexpr (!STATE) {
        // a warp's 32 channels of a token are 64 consecutive bytes
        int tlo, thi;
        inside(i * kC + 16 * qq, tlo, thi);
        const long long ld = (long long)p.hv * DV;
        const long long at = (S.ch.t0 + S.ch.m0 + i * kC + 16 * qq) * ld + tile * 128 + lrow;  // may be < 0
        __nv_bfloat16 ob[16];
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) {
          const float4 e = *reinterpret_cast<const float4*>(&S.eb[i % kSlots][hl][GDN_S(16 * qq + 4 * t4, kC - 3)]);
          const float2 ev[2] = {lo2(e), hi2(e)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = 4 * t4 + 2 * k;
            const float2 o = fma2(mul2(make_float2(o1[t], o1[t + 1]), make_float2(f1, f1)), ev[k],
                                  mul2(make_float2(o2[t], o2[t + 1]), make_float2(f2, f2)));
            const __nv_bfloat162 h = __floats2bfloat162_rn(o.x, o.y);
            ob[t] = h.x;
            ob[t + 1] = h.y;
          }
        }
        if (tlo <= 0 && thi >= 16) {
#pragma unroll
          for (int t = 0; t < 16; ++t) out[at + t * ld] = ob[t];
        } else {
#pragma unroll
          for (int t = 0; t < 16; ++t)
            if (t >= tlo && t < thi) out[at + t * ld] = ob[t];
        }
        // the block boundary at this chunk's end (a sequence that ends inside
        // the chunk does not reach it)
        if (i == next_ckpt) {
          const int kpc = p.ckpt_block / kC, ck_idx = S.ch.ck_idx + (i - S.ch.to_ckpt) / kpc;
          next_ckpt += kpc;
          if (ck_idx < p.max_ckpt && (i + 1) * kC <= S.ch.len - S.ch.m0) {
            const int32_t cid =
                GDN_GV(p.ckpt_ids, (long long)p.n_seq * p.max_ckpt)[(size_t)S.ch.n * p.max_ckpt + ck_idx];
            if (slot_class(cid, p.ck_num_slots) == 0) {
              // quarter rows, 32 bytes per access where the pool's alignment allows
              const auto to = GDN_GV(p.ck_ssm, p.ck_num_slots * slot_n) +
                              ((size_t)cid * slot_n + ((size_t)tile * 128 + lrow) * kDK + 32 * qq);
              if (((uintptr_t)p.ck_ssm & 31) == 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  st_global32(to.at(8 * e, 8), join4(st[4 * e], st[4 * e + 1]), join4(st[4 * e + 2], st[4 * e + 3]));
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) vec_at<float4>(to, 4 * e) = join4(st[2 * e], st[2 * e + 1]);
              }
            }
          }
        }
      }
    }
    if (named_sync_or(1, kCompute, !ok)) {
      if (tid == 0) report(p.err, GDN_DEV_ERR_TIMEOUT);
    } else if (STATE) {
      save(segs + ((S.ch.seg0 + S.ch.seg) * slot_n + (int64_t)tile0));
      if (qq == 0 && lrow % DV == 0)
        GDN_GV(a.seg_decay, (long long)a.n_segs * p.hv)[(S.ch.seg0 + S.ch.seg) * p.hv + h0 + hl] = seg_dec;
    } else if (S.ch.seg == S.ch.n_seg - 1) {
      save(GDN_GV(p.ssm, p.num_slots * slot_n) + ((size_t)S.ch.slot * slot_n + tile0));
    }
  }
  umma::fence_before();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(tmem, TM_COLS);
}

struct Layout {
  size_t rec, vhist, state, decay, total;
  int64_t n_chunks, n_segs;
  int32_t seg_chunks;
};
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Chunks per segment.  The lengths are on the device: the rule sees their sum.
//  * Enough chains for the SMs (sequences x tiles >= 96): whole sequences.  The
//    state pass costs about half as much again (8-group layer, in a graph,
//    whole and cut: 7 ragged sequences 126 and 134 us; 8 others of up to 1,931
//    tokens 187 and 194; 8 x 1000 135 and 142; 3 x 8192 401 and 552; 4 x 8192
//    417 and 668).
//  * Few chunks in all (16, or 24 of several sequences): whole too, since the
//    state pass costs more than it shortens (1 x 700 tokens 43 us whole, 58
//    cut; 1 x 1024 57 and 61; 1 x 1088 59 and 60; 1 x 1500 78 and 61; 2 x 768
//    48 and 60; 2 x 1000 60 and 62: two sequences break even near 32 chunks).
//  * Fewer chains: as many segments as fill the SMs, at most kMaxSegs per sequence
//    of the mean length (a segment reads all its predecessors' states), and
//    not below kMinSeg chunks.
constexpr int64_t kMinSeg = 8, kMaxSegs = 16;
int64_t seg_chunks(int64_t tiles, int64_t n_seq, int64_t total) {
  const int64_t chunks = (total + kC - 1) / kC, mean = (chunks + n_seq - 1) / n_seq;
  if (tiles * n_seq >= 96 || chunks <= (n_seq > 1 ? 24 : 16)) return 1 << 30;
  const int64_t fill = (tiles * chunks + sm_count() - 1) / sm_count();
  return max(max(fill + 1, kMinSeg), (mean + kMaxSegs - 1) / kMaxSegs);
}

Layout layout(const gdn_dims& d, int32_t n_seq, int64_t total) {
  Layout l;
  l.n_chunks = first_slot(total, n_seq);
  const int64_t tiles = (int64_t)d.hv * d.dv / 128;
  l.seg_chunks = (int32_t)seg_chunks(tiles, n_seq, total);
  l.n_segs = l.n_chunks / l.seg_chunks + n_seq;
  size_t off = 0;
  l.rec = off; off += sizeof(Record) * (size_t)l.n_chunks * d.hk;
  l.vhist = off; off += up256(sizeof(__nv_bfloat16) * 3 * (size_t)n_seq * d.hv * d.dv);
  l.state = off;
  if (l.seg_chunks < l.n_chunks) {
    off += sizeof(float) * (size_t)l.n_segs * d.hv * d.dv * d.dk;
    l.decay = off; off += up256(sizeof(float) * (size_t)l.n_segs * d.hv);
  } else {
    l.decay = off;
  }
  l.total = off + 1024;  // records start 1024-byte aligned
  return l;
}

// grid rows of the chain launch that hold the history work items
int64_t hist_blocks(int64_t C) { return (C + kThreads - 1) / kThreads; }
int64_t hist_rows(int64_t n_seq, int64_t C, int64_t tiles) { return (n_seq * hist_blocks(C) + tiles - 1) / tiles; }

template <int NH>
cudaError_t launch_chain(const ChunkArgs& a, const Layout& l, const CUtensorMap& xmap,
                         cudaStream_t s) {
  const size_t smem = sizeof(ChainSmem<NH>) + 1024;
  const unsigned tiles = (unsigned)(a.p.hv / NH);
  const dim3 grid(tiles, (unsigned)l.n_segs), all(tiles, (unsigned)(l.n_segs + hist_rows(a.p.n_seq, a.p.C, tiles)));
  cudaError_t e;
  if (l.seg_chunks < l.n_chunks) {
    constexpr auto k = ssm_chain_kernel<NH, true>;
    if ((e = ssm::allow_smem<k>(smem)) != cudaSuccess) return e;
    if ((e = launch_pdl(k, grid, dim3(kThreads), smem, s, dim3(1), a, xmap)) != cudaSuccess) return e;
  }
  constexpr auto k = ssm_chain_kernel<NH, false>;
  if ((e = ssm::allow_smem<k>(smem)) != cudaSuccess) return e;
  return launch_pdl(k, all, dim3(kThreads), smem, s, dim3(1), a, xmap);
}

}  // namespace

bool ssm_chunk_shape(const gdn_dims& d) {
  return d.dk == kDK && (d.dv == 64 || d.dv == 128) && (int64_t)(d.hv / d.hk) * d.dv % 128 == 0 && d.conv_width == 4 &&
         d.act_dtype == GDN_BF16 && d.conv_dtype == GDN_BF16;
}

bool ssm_chunk_supported(const gdn_dims& d, int32_t n_seq, int64_t total, const void* qkv, const void* out,
                         const gdn_ssm_params& p) {
  const int64_t tiles = (int64_t)d.hv * d.dv / 128;
  return ssm_chunk_shape(d) && total > 0 && d.hk <= 65535 &&
         layout(d, n_seq, total).n_segs + hist_rows(n_seq, channels(d), tiles) <= 65535 &&
         aligned(qkv, 16) && aligned(out, 16) && aligned(p.conv_w, 16);
}

size_t ssm_chunk_workspace(const gdn_dims& d, int32_t n_seq, int64_t total) { return layout(d, n_seq, total).total; }

cudaError_t ssm_chunk_launch(const ssm::PrefillArgs& p, const gdn_dims& d, void* ck_conv, void* workspace,
                             cudaStream_t s) {
  const Layout l = layout(d, p.n_seq, p.total);
  ChunkArgs a = {};
  a.p = p;
  uint8_t* const ws = reinterpret_cast<uint8_t*>(((uintptr_t)workspace + 1023) & ~(uintptr_t)1023);
  a.rec = reinterpret_cast<Record*>(ws + l.rec);
  a.vhist = reinterpret_cast<__nv_bfloat16*>(ws + l.vhist);
  a.seg_state = reinterpret_cast<float*>(ws + l.state);
  a.seg_decay = reinterpret_cast<float*>(ws + l.decay);
  a.n_chunks = (int32_t)l.n_chunks;
  a.n_segs = (int32_t)l.n_segs;
  a.seg_chunks = l.seg_chunks;
  // the features' walks: one wave of two CTAs per SM, so that all but a
  // walk's first chunk find their raw rows waiting
  a.feat_chunks = (int32_t)((l.n_chunks * p.hk + 2 * sm_count() - 1) / (2 * sm_count()));
  a.hist_blocks = (int32_t)hist_blocks(p.C);
  a.hist_groups = p.max_ckpt > pfx::kCkGroup ? (p.max_ckpt + pfx::kCkGroup - 1) / pfx::kCkGroup : 1;
  pfx::PrefillArgs& h = a.hist;
  h.ssm = p.ssm;
  h.conv = const_cast<void*>(p.conv);
  h.num_slots = p.num_slots;
  h.ck_ssm = p.ck_ssm;
  h.ck_conv = ck_conv;
  h.ck_num_slots = p.ck_num_slots;
  h.slot_ids = p.slot_ids;
  h.cu_seqlens = p.cu_seqlens;
  h.start_pos = p.start_pos;
  h.n_seq = p.n_seq;
  h.total = p.total;
  h.ckpt_ids = p.ckpt_ids;
  h.max_ckpt = p.max_ckpt;
  h.ckpt_block = p.ckpt_block;
  h.qkv = p.qkv;
  h.err = p.err;
  h.hk = p.hk;
  h.hv = p.hv;
  h.dk = p.dk;
  h.dv = p.dv;
  h.W = p.W;
  h.C = p.C;
  h.G = p.G;
  CUtensorMap xmap;
  cudaError_t e;
  if ((e = tensor_map_2d(&xmap, p.qkv, p.total, p.C, 2, 128, kRawRows, CU_TENSOR_MAP_SWIZZLE_NONE)) != cudaSuccess)
    return e;
  const size_t smem = sizeof(FeatSmem) + 1024;
  if ((e = ssm::allow_smem<ssm_features_kernel>(smem)) != cudaSuccess) return e;
  const unsigned walks = (unsigned)((l.n_chunks + a.feat_chunks - 1) / a.feat_chunks);
  if ((e = launch_pdl(ssm_features_kernel, dim3(walks + (unsigned)p.n_seq, (unsigned)p.hk), dim3(kFT), smem, s, dim3(1),
                      a, xmap)) != cudaSuccess)
    return e;
  return p.dv == 64 ? launch_chain<2>(a, l, xmap, s) : launch_chain<1>(a, l, xmap, s);
}

}  // namespace gdn
