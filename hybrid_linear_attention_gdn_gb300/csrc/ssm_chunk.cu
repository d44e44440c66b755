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
//   chain kernel's operand layouts (80 KB per chunk and group, read back
//   through L2 by the heads of the group, whose chains run side by side).
// chain kernel (128 V channels = one head of 128 or two of 64; sequence or
//   segment of one): walks its chunks in order, V rows in the tensor core's
//   M = 128 rows.  Per chunk, with S^T [dv][dk] in registers between chunks:
//     O1^T = S^T Q^T         tf32, S^T the A operand in TMEM
//     O2^T = V^T P^T         tf32, V^T the A operand in TMEM; two heads'
//                            P^T side by side (N = 128), each head's rows
//                            taken from its own half
//     dS^T = (V w)^T K       fp16 in two halves per operand (22 bits), three
//                            products, w_j = e^{b_last - b_j} dt_j
//     S^T <- e^{b_last} S^T + dS^T   fp32 on the CUDA cores, rounded to
//                            nearest: the tensor core's truncating
//                            accumulation never touches the long-lived state
//   Roundings: the two output products' operands to tf32 (2^-12 of their
//   terms, a tenth of the bf16 output's own 2^-9); the state's operands to
//   22 bits after a power-of-two scaling per chunk, by the largest |k| and
//   the largest |v w|, so that any input range keeps them.
// The work per 64 x 128 V values is bound by the instructions of the
// elementwise steps (conv + SiLU, P, operand conversion), not by the products
// or by memory.
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
// Sequence n's chunks occupy the slots from cu[n] / 64 + 2 n on: a sequence of
// len tokens touches at most len / 64 + 2 chunks, so the ranges are disjoint
// without a scan.  Its segments likewise: from that / seg_chunks + n on.
// One record per (chunk slot, group):
struct __align__(1024) Record {
  uint8_t q[4 * 64 * 128];    // q [token][dk] tf32, K-major swizzled, 32-column blocks of 8 KB
  uint8_t kh[128 * 128];      // k^T [dk][token] fp16, K-major swizzled: high halves
  uint8_t kl[128 * 128];      //   low halves
  uint8_t g[64 * 256];        // G [i][j] fp32, row i's 16-byte pieces p at p ^ (i & 7)
};
constexpr uint32_t kQBytes = sizeof(Record::q), kKBytes = 2 * sizeof(Record::kh), kGBytes = sizeof(Record::g);

struct ChunkArgs {
  PrefillArgs p;
  Record* rec;       // [chunk slots][hk]
  float* kscale;     // [chunk slots][hk]: 2^-e of the stored k
  float* seg_state;  // [segment slots][hv][dv][dk]
  float* seg_decay;  // [segment slots][hv]
  int32_t n_chunks, n_segs;  // slots
  int32_t seg_chunks;
};

__device__ __forceinline__ uint32_t f32_off(int r, int c, uint32_t blk) {
  return (uint32_t)(c >> 5) * blk + (uint32_t)(r >> 3) * 1024u + (uint32_t)(r & 7) * 128u +
         (uint32_t)((((c & 31) >> 2) ^ (r & 7)) << 4) + (uint32_t)(c & 3) * 4u;
}
__device__ __forceinline__ uint32_t g_off(int i, int c) {  // c a multiple of 4
  return (uint32_t)i * 256u + (uint32_t)(((c >> 2) ^ (i & 7)) << 4);
}

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
  s.first = s.t0 / kC + 2 * (int64_t)n;
  return s.len > 0;
}
// The last sequence whose first slot (first(n) = (cu[n] / 64 + 2 n) / div + n
// (div > 1) or cu[n] / 64 + 2 n (div 1)) is at most `slot`: one warp, 32
// candidates at a time.  Offsets outside [0, total] end the search early,
// never outside the array.
__device__ __forceinline__ int find_seq(const PrefillArgs& a, int64_t slot, int div, bool segs) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n_seq;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    bool le = false;
    if (i < n) {
      const int64_t c = (int64_t)cu[lo + i] / kC + 2 * (int64_t)(lo + i);
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
// bits of everything down to 2^-28 of m.  0 for m = 0, infinite or NaN.
__device__ __forceinline__ int scale_exp(uint32_t m_bits) {
  const int ex = (int)(m_bits >> 23);
  if (ex == 0 || ex == 255) return 0;
  const int e = 14 - (ex - 127);
  return e > 100 ? 100 : e;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// two values as fp16 high halves and the low halves that remain
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// ---------------------------------------------------------------------------
// features of q and k, G = Q K^T
// ---------------------------------------------------------------------------
// One CTA per (chunk slot, group), 256 threads: a channel pair and half of
// the chunk's tokens each.  HBM bound: 67 x 512 bytes in, 80 KB out.
constexpr int kFT = 256;
struct __align__(1024) FeatSmem {
  Record r;  // until G is done, r.kh and r.kl hold k [token][dk] tf32, as r.q
  uint32_t kmax;
};

// D += A B^T, one 16 x 8 tile of G by mma.sync tf32 (K = 8)
__device__ __forceinline__ void mma_g(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__global__ void __launch_bounds__(kFT, 2) ssm_features_kernel(const ChunkArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  FeatSmem& S = *reinterpret_cast<FeatSmem*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const PrefillArgs& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hq = blockIdx.y;
  const int64_t cslot = blockIdx.x;
  pdl_wait();
  const int n = find_seq(p, cslot, 1, false);
  Seq s;
  bool bad;
  if (!load_seq(p, n, s, bad) || slot_class(s.slot, p.num_slots)) return;
  const int64_t c = cslot - s.first;
  if (c < 0 || c >= s.nch) return;
  if (tid == 0) S.kmax = 0;
  const int64_t P = (s.p0 / kC + c) * kC;  // the chunk's first position
  const int cp = tid & 63;                 // channel pair of the part
  const bool isq = (tid & 64) == 0;
  const int half = tid >> 7;  // tokens 32 half ..
  const int ch = (isq ? hq : p.hk + hq) * kDK + 2 * cp;
  const auto qkv = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.qkv), p.total * p.C);
  const auto hist = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.conv), (long long)p.num_slots * 3 * p.C) +
                    (size_t)s.slot * 3 * p.C;
  const auto cw = GDN_GV(p.conv_w, (long long)p.C * 4);
  const float4 w0 = vec_at<const float4>(cw, (size_t)ch * 4), w1 = vec_at<const float4>(cw, (size_t)ch * 4 + 4);
  float2 bias = make_float2(0.f, 0.f);
  if (p.conv_bias) {
    const auto cb = GDN_GV(p.conv_bias, p.C);
    bias = make_float2(cb[ch], cb[ch + 1]);
  }
  // raw rows P + 32 half - 3 ..: inside the sequence from qkv, up to 3 before
  // it from the history, zeros elsewhere
  auto raw = [&](int64_t pos) -> float2 {
    const int64_t m = pos - s.p0;
    if (m >= 0 && m < s.len)
      return __bfloat1622float2(vec_at<const __nv_bfloat162>(qkv, (s.t0 + m) * p.C + ch));
    if (m < 0 && m >= -3) return __bfloat1622float2(vec_at<const __nv_bfloat162>(hist, (size_t)(3 + m) * p.C + ch));
    return make_float2(0.f, 0.f);
  };
  float2 y[32];
  float mx = 0.f;
  {
    const int64_t q0 = P + 32 * half;
    float2 x0 = raw(q0 - 3), x1 = raw(q0 - 2), x2 = raw(q0 - 1);
    float2 xr[32];
#pragma unroll
    for (int t = 0; t < 32; ++t) xr[t] = raw(q0 + t);
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      float2 acc = fma2(make_float2(w0.x, w1.x), x0, bias);
      acc = fma2(make_float2(w0.y, w1.y), x1, acc);
      acc = fma2(make_float2(w0.z, w1.z), x2, acc);
      acc = fma2(make_float2(w0.w, w1.w), xr[t], acc);
      const bool in = q0 + t >= s.p0 && q0 + t < s.p1;
      y[t] = in ? make_float2(silu_acc(acc.x), silu_acc(acc.y)) : make_float2(0.f, 0.f);
      x0 = x1;
      x1 = x2;
      x2 = xr[t];
      const float u = fabsf(y[t].x), v = fabsf(y[t].y);  // the finite ones
      mx = fmaxf(mx, fmaxf(u <= 3.4e38f ? u : 0.f, v <= 3.4e38f ? v : 0.f));
    }
  }
  pdl_trigger();
  static_assert(offsetof(Record, kl) == offsetof(Record, kh) + sizeof(Record::kh) && kKBytes == kQBytes, "k's place");
  uint8_t* const ktile = S.r.kh;
  uint8_t* const tile = isq ? S.r.q : ktile;
#pragma unroll
  for (int t = 0; t < 32; ++t)
    tile_at<float2>(tile, kQBytes, f32_off(32 * half + t, 2 * cp, 64 * 128)) =
        make_float2(umma::tf32_round(y[t].x), umma::tf32_round(y[t].y));
  __syncthreads();  // S.kmax cleared; the tiles written
  if (!isq) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
    if (lane == 0) atomicMax(&S.kmax, m);
  }
  // G: warp w rows 16 (w & 3) .., columns 32 (w >> 2) ..; above the diagonal
  // nothing is read
  {
    const int r0 = 16 * (warp & 3), c0 = 32 * (warp >> 2), gr = lane >> 2, gc = lane & 3;
    float d[4][4] = {};
    if (c0 < r0 + 16) {
#pragma unroll 4
      for (int k = 0; k < kDK; k += 8) {
        uint32_t av[4], bv[2];
        av[0] = tile_at<uint32_t>(S.r.q, kQBytes, f32_off(r0 + gr, k + gc, 64 * 128));
        av[1] = tile_at<uint32_t>(S.r.q, kQBytes, f32_off(r0 + gr + 8, k + gc, 64 * 128));
        av[2] = tile_at<uint32_t>(S.r.q, kQBytes, f32_off(r0 + gr, k + gc + 4, 64 * 128));
        av[3] = tile_at<uint32_t>(S.r.q, kQBytes, f32_off(r0 + gr + 8, k + gc + 4, 64 * 128));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          bv[0] = tile_at<uint32_t>(ktile, kQBytes, f32_off(c0 + 8 * t + gr, k + gc, 64 * 128));
          bv[1] = tile_at<uint32_t>(ktile, kQBytes, f32_off(c0 + 8 * t + gr, k + gc + 4, 64 * 128));
          mma_g(d[t], av, bv);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = r0 + gr + 8 * e, j = c0 + 8 * t + 2 * gc;
        tile_at<float2>(S.r.g, kGBytes, g_off(i, j & ~3) + (j & 3) * 4) = make_float2(d[t][2 * e], d[t][2 * e + 1]);
      }
  }
  __syncthreads();  // S.kmax complete, k read
  if (!isq) {
    const int e = scale_exp(S.kmax);
    const float f = exp2_int(e);
#pragma unroll
    for (int t8 = 0; t8 < 4; ++t8) {
      uint32_t h0[4], l0[4], h1[4], l1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = y[8 * t8 + 2 * i], v = y[8 * t8 + 2 * i + 1];
        split2(u.x * f, v.x * f, h0[i], l0[i]);
        split2(u.y * f, v.y * f, h1[i], l1[i]);
      }
      const uint32_t o0 = umma::sw128_off(2 * cp, 32 * half + 8 * t8, 0),
                     o1 = umma::sw128_off(2 * cp + 1, 32 * half + 8 * t8, 0);
      tile_at<uint4>(S.r.kh, sizeof(S.r.kh), o0) = make_uint4(h0[0], h0[1], h0[2], h0[3]);
      tile_at<uint4>(S.r.kl, sizeof(S.r.kl), o0) = make_uint4(l0[0], l0[1], l0[2], l0[3]);
      tile_at<uint4>(S.r.kh, sizeof(S.r.kh), o1) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
      tile_at<uint4>(S.r.kl, sizeof(S.r.kl), o1) = make_uint4(l1[0], l1[1], l1[2], l1[3]);
    }
    if (tid == 64) GDN_GV(a.kscale, (long long)a.n_chunks * p.hk)[cslot * p.hk + hq] = exp2_int(-e);
  }
  umma::fence_proxy_async();
  __syncthreads();
  if (tid == 0) {
    const int64_t ri = cslot * p.hk + hq;
    if (GDN_SPAN_G(ri, 1, (long long)a.n_chunks * p.hk)) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(a.rec + ri),
                   "r"(smem_addr(&S.r)), "r"((uint32_t)sizeof(Record))
                   : "memory");
      bulk_commit();
      bulk_wait_all();
    }
  }
}

// ---------------------------------------------------------------------------
// the chain
// ---------------------------------------------------------------------------
constexpr int kThreads = 512;

// TMEM columns
constexpr uint32_t TM_S = 0;     // S^T (operand), then dS^T
constexpr uint32_t TM_O1 = 128;  // [dv rows][64 tokens]
constexpr uint32_t TM_O2 = 192;  // [dv rows][64 tokens of each head]
constexpr uint32_t TM_V = 320;   // V^T tf32 [dv rows][64 tokens]
constexpr uint32_t TM_WH = 384;  // (V w)^T fp16 pairs: high halves, 32 columns
constexpr uint32_t TM_WL = 416;  //   low halves
constexpr uint32_t TM_COLS = 512;

template <int NH>
struct __align__(1024) ChainSmem {
  uint8_t q[kQBytes];
  uint8_t k[kKBytes];
  uint8_t pt[2 * NH * 64 * 128];  // P [head, i][j] tf32: two 32-column blocks
  uint8_t g[kGBytes];
  __nv_bfloat16 raw[kRawRows][128];
  __align__(16) __nv_bfloat16 ot[kC][128];
  // per chunk parity and head
  float b2[2][NH][kC];   // b log2(e)
  float eb[2][NH][kC];   // e^b
  float dt[2][NH][kC];
  float w[2][NH][kC];    // e^{b_last - b} dt
  float dec[2][NH];      // e^{b_last}
  uint32_t vmax[2];
  uint64_t x_bar, q_bar, k_bar, g_bar, o1_bar, mma_bar;
  uint32_t tmem_base;
  int seq;
};

// 8 consecutive columns of this thread's TMEM lane, written
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8], int line = __builtin_LINE()) {
  if (!umma::tmem_ok(taddr, 8, true, line)) return;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
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
    ssm_chain_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap xmap,
                     const __grid_constant__ CUtensorMap omap) {
  constexpr int DV = 128 / NH;
  using SM = ChainSmem<NH>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  SM& S = *reinterpret_cast<SM*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const PrefillArgs& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile = blockIdx.x, h0 = tile * NH, hq = h0 / p.G;
  pdl_wait();
  if (warp == 0) {
    const int f = find_seq(p, blockIdx.y, a.seg_chunks, true);
    if (lane == 0) S.seq = f;
  }
  __syncthreads();
  const int n = S.seq;
  Seq s;
  bool bad_seq;
  const bool some = load_seq(p, n, s, bad_seq);
  const int64_t seg_first = (s.t0 / kC + 2 * (int64_t)n) / a.seg_chunks + n;
  const int seg = bad_seq ? 0 : (int)(blockIdx.y - seg_first);
  // sequences with errors, padded or empty ones are dealt with by their own
  // first segment slot
  if (bad_seq || !some || slot_class(s.slot, p.num_slots)) {
    return;  // reported and zeroed by ssm_check_kernel
  }
  const int n_seg = (s.nch + a.seg_chunks - 1) / a.seg_chunks;
  if (seg < 0 || seg >= n_seg || (STATE && seg == n_seg - 1)) return;
  const int c_begin = seg * a.seg_chunks, c_end = min(s.nch, c_begin + a.seg_chunks);

  if (warp == 0) umma::tmem_alloc(&S.tmem_base, TM_COLS);
  if (tid == 0) {
    mbar_init(&S.x_bar, 1);
    mbar_init(&S.q_bar, 1);
    mbar_init(&S.k_bar, 1);
    mbar_init(&S.g_bar, 1);
    mbar_init(&S.o1_bar, 1);
    mbar_init(&S.mma_bar, 1);
    S.vmax[0] = S.vmax[1] = 0;
    fence_mbar_init();
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = S.tmem_base;
  const int lrow = 32 * (warp & 3) + lane;  // V channel of the tile, TMEM lane
  const int qq = warp >> 2;                 // token (or dk column) quarter
  const int hl = lrow / DV;                 // this row's head within the tile
  const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const int ch = 2 * p.hk * kDK + tile * 128 + lrow;

  // loads of chunk c, by thread 0
  const int64_t rec0 = (s.first * p.hk) + hq;
  auto bulk = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, bytes);
    if (GDN_GBYTES(src, bytes, a.rec, (long long)a.n_chunks * p.hk * sizeof(Record)) && GDN_SBYTES(dst, bytes, S))
      bulk_g2s(dst, src, bytes, bar);
  };
  int n_x = 0, n_q = 0, n_k = 0, n_g = 0;  // issued (thread 0)
  auto load_x = [&](int c) {
    const int32_t row0 = (int32_t)(s.t0 + ((s.p0 / kC + c) * kC - 3 - s.p0));  // may be < 0: zeros
    mbar_arrive_expect_tx(&S.x_bar, (uint32_t)sizeof(S.raw));
    if (GDN_SPAN_G(2 * p.hk * kDK + tile * 128, 128, p.C) && GDN_SBYTES(&S.raw[0][0], sizeof(S.raw), S))
      tma_load_2d(&S.raw[0][0], &xmap, 2 * p.hk * kDK + tile * 128, row0, &S.x_bar);
    ++n_x;
  };
  auto load_q = [&](int c) { bulk(S.q, a.rec[rec0 + (int64_t)c * p.hk].q, kQBytes, &S.q_bar); ++n_q; };
  auto load_k = [&](int c) { bulk(S.k, a.rec[rec0 + (int64_t)c * p.hk].kh, kKBytes, &S.k_bar); ++n_k; };
  auto load_g = [&](int c) { bulk(S.g, a.rec[rec0 + (int64_t)c * p.hk].g, kGBytes, &S.g_bar); ++n_g; };

  // gates of chunk c into buffer buf: warp 8 + head; two tokens per lane,
  // their logits loaded one chunk ahead
  const bool gate_warp = warp >= 8 && warp < 8 + NH;
  const int gh = h0 + (gate_warp ? warp - 8 : 0);
  const auto gate_a = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.a), p.total * p.hv);
  float ga[2] = {0.f, 0.f};
  auto gate_load = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = (s.p0 / kC + c) * kC + 32 * i + lane - s.p0;
      ga[i] = c < c_end && m >= 0 && m < s.len ? __bfloat162float(gate_a[(s.t0 + m) * p.hv + gh]) : 0.f;
    }
  };
  const float A_log = GDN_GV(p.A_log, p.hv)[gh], dtb = GDN_GV(p.dt_bias, p.hv)[gh];
  auto gates = [&](int c, int buf) {
    float dt[2], g[2], b[2], suf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = (s.p0 / kC + c) * kC + 32 * i + lane - s.p0;
      const bool in = m >= 0 && m < s.len;
      const Gate t = gate(A_log, dtb, ga[i]);
      dt[i] = in ? t.dt : 0.f;
      g[i] = in ? floor_log_decay(t.g) : 0.f;
      b[i] = suf[i] = g[i];
    }
    gate_load(c + 1);
    // inclusive sums from the front and from the back: e^{b_last - b_j} from
    // its own sum, exact to its own size whatever b_last is
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float u = __shfl_up_sync(0xffffffffu, b[i], o), v = __shfl_down_sync(0xffffffffu, suf[i], o);
        if (lane >= o) b[i] += u;
        if (lane + o < 32) suf[i] += v;
      }
    }
    b[1] += __shfl_sync(0xffffffffu, b[0], 31);
    const float back = __shfl_sync(0xffffffffu, suf[1], 0), all = back + __shfl_sync(0xffffffffu, suf[0], 0);
    const float nx = __shfl_down_sync(0xffffffffu, suf[0], 1), ny = __shfl_down_sync(0xffffffffu, suf[1], 1);
    suf[0] = (lane < 31 ? nx : 0.f) + back;
    suf[1] = lane < 31 ? ny : 0.f;
    const int hh = warp - 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 32 * i + lane;
      S.b2[buf][hh][t] = b[i] * 1.4426950408889634f;
      S.eb[buf][hh][t] = expf(b[i]);
      S.dt[buf][hh][t] = dt[i];
      S.w[buf][hh][t] = expf(suf[i]) * dt[i];
    }
    if (lane == 0) S.dec[buf][hh] = expf(all);
  };

  // the state entering the segment, S^T row lrow, columns 32 qq ..
  float st[32];
  float seg_dec = 1.f;
  const size_t tile_off = ((size_t)tile * 128 + lrow) * kDK + 32 * qq;  // within one slot's [hv][dv][dk]
  const long long slot_n = (long long)p.hv * DV * kDK;
  const auto segs = GDN_GV(a.seg_state, a.n_segs * slot_n);
  const auto pool = GDN_GV(p.ssm, p.num_slots * slot_n) + ((size_t)s.slot * slot_n + tile_off);
  {
    // one segment: from the slot.  Several: the first launch starts the first
    // segment from the slot, keeping a copy at the (otherwise unused) last
    // segment's place for the second launch, and the others from zero
    const auto keep = segs + ((n_seg > 1 ? (seg_first + n_seg - 1) * slot_n : 0) + (n_seg > 1 ? tile_off : 0));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (seg == 0) {
        if (STATE || n_seg == 1) v = vec_at<const float4>(pool, 4 * i);
        else v = vec_at<const float4>(keep, 4 * i);
        if (STATE) vec_at<float4>(keep, 4 * i) = v;
      }
      st[4 * i] = v.x; st[4 * i + 1] = v.y; st[4 * i + 2] = v.z; st[4 * i + 3] = v.w;
    }
    if (!STATE) {
      for (int k = 0; k < seg; ++k) {
        const auto L = segs + ((seg_first + k) * slot_n + tile_off);
        const float d = k ? GDN_GV(a.seg_decay, (long long)a.n_segs * p.hv)[(seg_first + k) * p.hv + h0 + hl] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 v = vec_at<const float4>(L, 4 * i);
          st[4 * i] = fmaf(d, st[4 * i], v.x);
          st[4 * i + 1] = fmaf(d, st[4 * i + 1], v.y);
          st[4 * i + 2] = fmaf(d, st[4 * i + 2], v.z);
          st[4 * i + 3] = fmaf(d, st[4 * i + 3], v.w);
        }
      }
    }
  }
  auto put_state = [&]() {  // the operand S^T
    float r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = umma::tf32_round(st[i]);
    umma::tmem_st32(tlane + TM_S + 32 * qq, r);
  };
  if (tid == 0) {
    load_x(c_begin);
    load_k(c_begin);
    if (!STATE) {
      load_q(c_begin);
      load_g(c_begin);
    }
  }
  if (gate_warp) {
    gate_load(c_begin);
    gates(c_begin, c_begin & 1);
  }
  const float4 w4 = vec_at<const float4>(GDN_GV(p.conv_w, (long long)p.C * 4), (size_t)ch * 4);
  const float bias = p.conv_bias ? GDN_GV(p.conv_bias, p.C)[ch] : 0.f;
  // P's rows of this thread: row pr of the heads' 64 NH, PC columns from pc;
  // what lies above the diagonal stays zero
  constexpr int PC = 8 * NH;
  const int pr = NH == 2 ? lrow : (lrow & 63), pi = pr & 63, ph = pr >> 6;
  const int pc = 16 * qq + (NH == 2 ? 0 : 8 * (lrow >> 6));
  const float skip = p.D ? GDN_GV(p.D, p.hv)[h0 + ph] : 0.f;
  constexpr uint32_t kPBlk = NH * 64 * 128;
  if (!STATE) {
    put_state();
#pragma unroll
    for (int c4 = 0; c4 < PC / 4; ++c4)
      tile_at<float4>(S.pt, sizeof(S.pt), f32_off(pr, pc + 4 * c4, kPBlk)) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int kpc = p.ckpt_block / kC;
  const int q0 = (int)((s.p0 / kC) % kpc);
  auto ckpt_slot = [&](int c) -> int32_t {  // checkpoint slot at the end of chunk c, -1: none
    if (c == s.nch - 1 && s.p1 % kC) return -1;
    const int q = q0 + c + 1;
    if (q % kpc) return -1;
    const int idx = q / kpc - 1;
    if (idx >= p.max_ckpt) return -1;
    const int32_t id = GDN_GV(p.ckpt_ids, (long long)p.n_seq * p.max_ckpt)[(size_t)n * p.max_ckpt + idx];
    return slot_class(id, p.ck_num_slots) == 0 ? id : -1;
  };
  constexpr uint32_t ID_O1 = umma::idesc_tf32(128, kC, false, false);
  constexpr uint32_t ID_O2 = umma::idesc_tf32(128, NH * kC, false, false);
  constexpr uint32_t ID_S = umma::idesc_f16(128, kDK, false, false);
  static_assert(TM_O1 == TM_S + kDK && TM_O2 == TM_O1 + kC && TM_V == TM_O2 + 2 * kC && TM_WH == TM_V + kC &&
                    TM_WL == TM_WH + kC / 2 && TM_WL + kC / 2 <= TM_COLS,
                "TMEM regions");

  bool bad = false;
  int n_o1 = 0, n_mma = 0;  // committed (thread 0)
  umma::fence_before();
  __syncthreads();
  int c = c_begin;
  for (; c < c_end; ++c) {
    const int it = c - c_begin, buf = c & 1;
    const uint32_t par = it & 1;
    const int64_t P = (s.p0 / kC + c) * kC;
    const int tlo = (int)max((int64_t)0, min((int64_t)kC, s.p0 - P));
    const int thi = (int)max((int64_t)0, min((int64_t)kC, s.p1 - P));
    // O1^T = S^T Q^T
    if (!STATE && tid == 0) {
      if (mbar_wait(&S.q_bar, par)) {
        umma::fence_after();
        const uint64_t dq = umma::desc(smem_addr(S.q), 16, 1024);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          umma::mma_tf32_ta(tmem + TM_O1, tmem + TM_S + 8 * k, umma::adv(dq, (k >> 2) * 8192 + (k & 3) * 32), ID_O1,
                            k > 0);
        umma::commit(&S.o1_bar);
        ++n_o1;
      } else {
        bad = true;
      }
    }
    // v: conv1d + SiLU of channel lrow, tokens 16 qq ..
    if (!mbar_wait(&S.x_bar, par)) bad = true;
    if (P - 3 < s.p0) {
      // the up to 3 rows just before the sequence come from the history
      const int64_t lo = max(P - 3, s.p0 - 3), hi = min(P + kC, s.p0);
      const auto hist = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.conv), (long long)p.num_slots * 3 * p.C) +
                        (size_t)s.slot * 3 * p.C;
      for (int64_t pos = lo; pos < hi; ++pos)
        if (tid < 128) S.raw[GDN_S((int)(pos - (P - 3)), kRawRows)][tid] =
            hist[(size_t)(3 - (s.p0 - pos)) * p.C + 2 * p.hk * kDK + tile * 128 + tid];
      umma::fence_proxy_async();  // before the next chunk's copy into these rows
      __syncthreads();
    }
    float y[16];
    {
      const auto xs = GDN_SV(&S.raw[0][0], kRawRows * 128) + (16 * qq * 128 + lrow);
      float x[19];
#pragma unroll
      for (int r = 0; r < 19; ++r) x[r] = __bfloat162float(xs[r * 128]);
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        float acc = fmaf(w4.x, x[t], bias);
        acc = fmaf(w4.y, x[t + 1], acc);
        acc = fmaf(w4.z, x[t + 2], acc);
        acc = fmaf(w4.w, x[t + 3], acc);
        const bool in = (unsigned)(16 * qq + t - tlo) < (unsigned)(thi - tlo);
        y[t] = in ? silu_acc(acc) : 0.f;
      }
    }
    if (!STATE) {
      float r[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) r[t] = umma::tf32_round(y[t]);
      __syncwarp();
      umma::tmem_st16(tlane + TM_V + 16 * qq, r);
    }
    // V w and its largest magnitude
    {
      uint32_t m = 0;
      const auto ws = GDN_SV(&S.w[buf][hl][0], kC);
#pragma unroll
      for (int t4 = 0; t4 < 4; ++t4) {
        const float4 v = vec_at<const float4>(ws, 16 * qq + 4 * t4);
        y[4 * t4] *= v.x; y[4 * t4 + 1] *= v.y; y[4 * t4 + 2] *= v.z; y[4 * t4 + 3] *= v.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(y[4 * t4 + i]) & 0x7fffffffu);
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) atomicMax(&S.vmax[buf], m);
    }
    // P from G
    if (!STATE) {
      if (!mbar_wait(&S.g_bar, par)) bad = true;
      if (pc <= pi) {
        const float bi = S.b2[buf][ph][pi];
#pragma unroll
        for (int c4 = 0; c4 < PC / 4; ++c4) {
          const int j = pc + 4 * c4;
          const float4 gv = tile_at<float4>(S.g, sizeof(S.g), g_off(pi, j));
          const float4 bj = *reinterpret_cast<const float4*>(&S.b2[buf][ph][GDN_S(j, kC - 3)]);
          const float4 dj = *reinterpret_cast<const float4*>(&S.dt[buf][ph][j]);
          float e[4] = {bi - bj.x, bi - bj.y, bi - bj.z, bi - bj.w};
          const float gd[4] = {gv.x * dj.x, gv.y * dj.y, gv.z * dj.z, gv.w * dj.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x;
            asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(x) : "f"(e[i]));
            x *= gd[i];
            if (j + i == pi) x += skip;
            e[i] = j + i <= pi ? umma::tf32_round(x) : 0.f;
          }
          tile_at<float4>(S.pt, sizeof(S.pt), f32_off(pr, j, kPBlk)) = make_float4(e[0], e[1], e[2], e[3]);
        }
      }
    }
    if (__syncthreads_or(bad)) break;  // #1: raw rows and G read, the maximum complete
    if (tid == 0 && c + 1 < c_end) {
      load_x(c + 1);
      if (!STATE) load_g(c + 1);
    }
    if (tid == 32) S.vmax[buf ^ 1] = 0;
    if (S.vmax[buf] >= 0x7f800000u) {
      // infinite or NaN values among V w: the scale of the finite ones
      __syncthreads();
      if (tid == 0) S.vmax[buf] = 0;
      __syncthreads();
      uint32_t m = 0;
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const uint32_t u = __float_as_uint(y[t]) & 0x7fffffffu;
        m = max(m, u < 0x7f800000u ? u : 0u);
      }
      atomicMax(&S.vmax[buf], m);
      __syncthreads();
    }
    const int ve = scale_exp(S.vmax[buf]);
    __syncwarp();
    {
      const float f = exp2_int(ve);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) split2(y[2 * t] * f, y[2 * t + 1] * f, hi[t], lo[t]);
      tmem_st8(tlane + TM_WH + 8 * qq, hi);
      tmem_st8(tlane + TM_WL + 8 * qq, lo);
    }
    if (gate_warp && c + 1 < c_end) gates(c + 1, buf ^ 1);
    if (!STATE && tid == 0) bulk_wait_read();  // the output staging has been read
    umma::fence_proxy_async();
    umma::fence_before();
    __syncthreads();  // #2: operands complete
    if (tid == 0) {
      // dS^T takes the place of S^T, which O1's product has read by then
      if (!STATE && !mbar_wait(&S.o1_bar, par)) bad = true;
      if (!mbar_wait(&S.k_bar, par)) bad = true;
      if (!bad) {
        umma::fence_after();
        if (!STATE) {
          const uint64_t dp = umma::desc(smem_addr(S.pt), 16, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma::mma_tf32_ta(tmem + TM_O2, tmem + TM_V + 8 * k, umma::adv(dp, (k >> 2) * kPBlk + (k & 3) * 32),
                              ID_O2, k > 0);
        }
        const uint64_t dh = umma::desc(smem_addr(S.k), 16, 1024);
        const uint64_t dl = umma::adv(dh, sizeof(Record::kh));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16_ta(tmem + TM_S, tmem + TM_WL + 8 * k, umma::adv(dh, 32 * k), ID_S, k > 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16_ta(tmem + TM_S, tmem + TM_WH + 8 * k, umma::adv(dl, 32 * k), ID_S, true);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16_ta(tmem + TM_S, tmem + TM_WH + 8 * k, umma::adv(dh, 32 * k), ID_S, true);
        umma::commit(&S.mma_bar);
        ++n_mma;
        if (!STATE && c + 1 < c_end) load_q(c + 1);
      }
    }
    const float kscale = GDN_GV(a.kscale, (long long)a.n_chunks * p.hk)[(s.first + c) * p.hk + hq];
    if (!mbar_wait(&S.mma_bar, par)) bad = true;
    __syncwarp();
    umma::fence_after();
    if (tid == 0 && !bad && c + 1 < c_end) load_k(c + 1);
    __syncwarp();
    // the state after the chunk
    {
      const float dec = S.dec[buf][hl], f = exp2_int(-ve);
      seg_dec *= dec;
      float d[32];
      umma::tmem_ld32(tlane + TM_S + 32 * qq, d);
#pragma unroll
      for (int i = 0; i < 32; ++i) st[i] = fmaf(st[i], dec, d[i] * kscale * f);
    }
    if constexpr (!STATE) {
      float o1[16], o2[16];
      umma::tmem_ld16(tlane + TM_O1 + 16 * qq, o1);
      umma::tmem_ld16(tlane + TM_O2 + (NH == 2 ? hl * kC : 0) + 16 * qq, o2);
      put_state();
      const auto ot = GDN_SV(&S.ot[0][0], kC * 128);
#pragma unroll
      for (int t4 = 0; t4 < 4; ++t4) {
        const float4 e = *reinterpret_cast<const float4*>(&S.eb[buf][hl][GDN_S(16 * qq + 4 * t4, kC - 3)]);
        const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ot[(16 * qq + 4 * t4 + i) * 128 + lrow] = __float2bfloat16_rn(fmaf(o1[4 * t4 + i], ev[i], o2[4 * t4 + i]));
      }
      const int32_t cid = ckpt_slot(c);
      if (cid >= 0) {
        const auto K = GDN_GV(p.ck_ssm, p.ck_num_slots * slot_n) + ((size_t)cid * slot_n + tile_off);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          vec_at<float4>(K, 4 * i) = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
      }
      umma::fence_proxy_async();
    }
    umma::fence_before();
    if (__syncthreads_or(bad)) break;  // #3: the output staged, S^T in place, TMEM read
    if constexpr (!STATE) {
      const auto ot = GDN_SV(&S.ot[0][0], kC * 128);
      if (thi - tlo == kC) {
        if (tid == 0 && GDN_SPAN_G(s.t0 + (P - s.p0), kC, p.total)) {
          tma_store_2d(&omap, &S.ot[0][0], tile * 128, (int32_t)(s.t0 + (P - s.p0)));
          bulk_commit();
        }
      } else {
        const auto out = GDN_GV(reinterpret_cast<__nv_bfloat16*>(p.out), p.total * p.hv * DV);
        for (int e = tid; e < kC * 16; e += kThreads) {
          const int r = e >> 4, piece = e & 15;
          if (r >= tlo && r < thi)
            vec_at<uint4>(out, ((s.t0 + P - s.p0 + r) * p.hv) * DV + tile * 128 + 8 * piece) =
                vec_at<const uint4>(ot, r * 128 + 8 * piece);
        }
      }
    }
  }
  if (c < c_end) {
    // a wait expired: let what is in flight land before the memory goes away
    if (tid == 0) {
      report(p.err, GDN_DEV_ERR_TIMEOUT);
      for (int k = max(0, n_x - 1); k < n_x; ++k) mbar_wait(&S.x_bar, k & 1);
      for (int k = max(0, n_q - 1); k < n_q; ++k) mbar_wait(&S.q_bar, k & 1);
      for (int k = max(0, n_k - 1); k < n_k; ++k) mbar_wait(&S.k_bar, k & 1);
      for (int k = max(0, n_g - 1); k < n_g; ++k) mbar_wait(&S.g_bar, k & 1);
      if (n_o1) mbar_wait(&S.o1_bar, (n_o1 - 1) & 1);
      if (n_mma) mbar_wait(&S.mma_bar, (n_mma - 1) & 1);
    }
  } else if (STATE) {
    const auto L = segs + ((seg_first + seg) * slot_n + tile_off);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      vec_at<float4>(L, 4 * i) = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
    if (qq == 0 && lrow % DV == 0)
      GDN_GV(a.seg_decay, (long long)a.n_segs * p.hv)[(seg_first + seg) * p.hv + h0 + hl] = seg_dec;
  } else if (seg == n_seg - 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      vec_at<float4>(pool, 4 * i) = make_float4(st[4 * i], st[4 * i + 1], st[4 * i + 2], st[4 * i + 3]);
  }
  if (tid == 0) bulk_wait_all();
  umma::fence_before();
  __syncthreads();
  if (warp == 0) umma::tmem_dealloc(tmem, TM_COLS);
}

// Inconsistent sequences reported, unusable slots' rows zeroed (grid: sequences).
__global__ void __launch_bounds__(256) ssm_check_kernel(const PrefillArgs p) {
  pdl_wait();
  pdl_trigger();
  const int n = blockIdx.x;
  Seq s;
  bool bad;
  const bool some = load_seq(p, n, s, bad);
  if (bad && threadIdx.x == 0) report(p.err, GDN_DEV_ERR_SEQLENS);
  const int cls = slot_class(s.slot, p.num_slots);
  if (!bad && cls == 2 && threadIdx.x == 0) report(p.err, GDN_DEV_ERR_SLOT_OOB);
  if (!some || !cls) return;
  const auto out = GDN_GV(reinterpret_cast<uint4*>(p.out), p.total * p.hv * p.dv / 8);
  const int64_t row = (int64_t)p.hv * p.dv / 8;
  for (int64_t e = threadIdx.x; e < s.len * row; e += blockDim.x) out[s.t0 * row + e] = make_uint4(0u, 0u, 0u, 0u);
}

struct Layout {
  size_t rec, kscale, state, decay, total;
  int64_t n_chunks, n_segs;
  int32_t seg_chunks;
};
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

Layout layout(const gdn_dims& d, int32_t n_seq, int64_t total) {
  Layout l;
  l.n_chunks = total / kC + 2 * (int64_t)n_seq;
  const int64_t tiles = (int64_t)d.hv * d.dv / 128;
  l.seg_chunks = 1 << 30;
  (void)tiles;
  l.n_segs = l.n_chunks / l.seg_chunks + n_seq;
  size_t off = 0;
  l.rec = off; off += sizeof(Record) * (size_t)l.n_chunks * d.hk;
  l.kscale = off; off += up256(sizeof(float) * (size_t)l.n_chunks * d.hk);
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

template <int NH>
cudaError_t launch_chain(const ChunkArgs& a, const Layout& l, const CUtensorMap& xmap, const CUtensorMap& omap,
                         cudaStream_t s) {
  const size_t smem = sizeof(ChainSmem<NH>) + 1024;
  const dim3 grid((unsigned)(a.p.hv / NH), (unsigned)l.n_segs);
  cudaError_t e;
  if (l.seg_chunks < l.n_chunks) {
    auto k = ssm_chain_kernel<NH, true>;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
    if ((e = launch_plain(k, grid, dim3(kThreads), smem, s, dim3(1), a, xmap, omap)) != cudaSuccess) return e;
  }
  auto k = ssm_chain_kernel<NH, false>;
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
  return launch_plain(k, grid, dim3(kThreads), smem, s, dim3(1), a, xmap, omap);
}

}  // namespace

bool ssm_chunk_shape(const gdn_dims& d) {
  return d.dk == kDK && (d.dv == 64 || d.dv == 128) && (int64_t)(d.hv / d.hk) * d.dv % 128 == 0 && d.conv_width == 4 &&
         d.act_dtype == GDN_BF16 && d.conv_dtype == GDN_BF16;
}

bool ssm_chunk_supported(const gdn_dims& d, int32_t n_seq, int64_t total, const void* qkv, const void* out,
                         const gdn_ssm_params& p) {
  return ssm_chunk_shape(d) && total > 0 && layout(d, n_seq, total).n_segs <= 65535 && d.hk <= 65535 &&
         aligned(qkv, 16) && aligned(out, 16) && aligned(p.conv_w, 16);
}

size_t ssm_chunk_workspace(const gdn_dims& d, int32_t n_seq, int64_t total) { return layout(d, n_seq, total).total; }

cudaError_t ssm_chunk_launch(const ssm::PrefillArgs& p, const gdn_dims& d, void* workspace, cudaStream_t s) {
  const Layout l = layout(d, p.n_seq, p.total);
  ChunkArgs a = {};
  a.p = p;
  uint8_t* const ws = reinterpret_cast<uint8_t*>(((uintptr_t)workspace + 1023) & ~(uintptr_t)1023);
  a.rec = reinterpret_cast<Record*>(ws + l.rec);
  a.kscale = reinterpret_cast<float*>(ws + l.kscale);
  a.seg_state = reinterpret_cast<float*>(ws + l.state);
  a.seg_decay = reinterpret_cast<float*>(ws + l.decay);
  a.n_chunks = (int32_t)l.n_chunks;
  a.n_segs = (int32_t)l.n_segs;
  a.seg_chunks = l.seg_chunks;
  CUtensorMap xmap, omap;
  cudaError_t e;
  if ((e = tensor_map_2d(&xmap, p.qkv, p.total, p.C, 2, 128, kRawRows, CU_TENSOR_MAP_SWIZZLE_NONE)) != cudaSuccess)
    return e;
  if ((e = tensor_map_2d(&omap, p.out, p.total, (int64_t)p.hv * p.dv, 2, 128, kC, CU_TENSOR_MAP_SWIZZLE_NONE)) !=
      cudaSuccess)
    return e;
  const size_t smem = sizeof(FeatSmem) + 1024;
  if ((e = cudaFuncSetAttribute(ssm_features_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
      cudaSuccess)
    return e;
  if ((e = launch_plain(ssm_features_kernel, dim3((unsigned)l.n_chunks, (unsigned)p.hk), dim3(kFT), smem, s, dim3(1),
                        a)) != cudaSuccess)
    return e;
  if ((e = launch_plain(ssm_check_kernel, dim3((unsigned)p.n_seq), dim3(256), 0, s, dim3(1), p)) != cudaSuccess)
    return e;
  return p.dv == 64 ? launch_chain<2>(a, l, xmap, omap, s) : launch_chain<1>(a, l, xmap, omap, s);
}

}  // namespace gdn
