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
// the chunk's tokens each.  HBM bound: 67 x 512 bytes in, 80 KB out.  q and k
// stand one above the other as one 128-row operand, so that one product of
// M = 128 gives G in its upper half; k's place then takes its fp16 halves.
constexpr int kFT = 256;
struct __align__(1024) FeatSmem {
  uint8_t qk[4 * 128 * 128];  // [q; k] tf32, K-major swizzled, 32-column blocks of 16 KB; then in
                              // the k halves of the blocks: kh rows 0.., 64.., kl rows 0.., 64..
  uint8_t g[kGBytes];
  uint64_t bar;
  uint32_t kmax, tmem_base;
};

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(smem_addr(src)),
               "r"(bytes)
               : "memory");
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
  if (warp == 0) umma::tmem_alloc(&S.tmem_base, 64);
  if (tid == 0) {
    S.kmax = 0;
    mbar_init(&S.bar, 1);
    fence_mbar_init();
  }
  const int64_t P = (s.p0 / kC + c) * kC;  // the chunk's first position
  const int cp = tid & 63;                 // channel pair of the part
  const bool isq = (tid & 64) == 0;        // warps 0, 1, 4, 5
  const int half = tid >> 7;               // tokens 32 half ..
  const int ch = (isq ? hq : p.hk + hq) * kDK + 2 * cp;
  const auto qkv = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.qkv), p.total * p.C);
  const auto cw = GDN_GV(p.conv_w, (long long)p.C * 4);
  const float4 w0 = vec_at<const float4>(cw, (size_t)ch * 4), w1 = vec_at<const float4>(cw, (size_t)ch * 4 + 4);
  float2 bias = make_float2(0.f, 0.f);
  if (p.conv_bias) {
    const auto cb = GDN_GV(p.conv_bias, p.C);
    bias = make_float2(cb[ch], cb[ch + 1]);
  }
  // raw rows from 3 before the thread's first token: of the sequence, of the
  // history (up to 3 before the sequence), zeros elsewhere
  const int64_t m0 = P + 32 * half - s.p0;  // the first token's index in the sequence
  const bool full = m0 >= 3 && m0 + 32 <= s.len;
  __nv_bfloat162 xr[35];
  if (full) {
    const auto src = qkv + (s.t0 + m0 - 3) * p.C + ch;
#pragma unroll
    for (int r = 0; r < 35; ++r) xr[r] = vec_at<const __nv_bfloat162>(src, (size_t)r * p.C);
  } else {
    const auto hist = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.conv), (long long)p.num_slots * 3 * p.C) +
                      (size_t)s.slot * 3 * p.C;
#pragma unroll
    for (int r = 0; r < 35; ++r) {
      const int64_t m = m0 - 3 + r;
      xr[r] = __floats2bfloat162_rn(0.f, 0.f);
      if (m >= 0 && m < s.len) xr[r] = vec_at<const __nv_bfloat162>(qkv, (s.t0 + m) * p.C + ch);
      else if (m < 0 && m >= -3) xr[r] = vec_at<const __nv_bfloat162>(hist, (size_t)(3 + m) * p.C + ch);
    }
  }
  float2 y[32];
  float mx = 0.f;
  {
    const float2 v0 = make_float2(w0.x, w1.x), v1 = make_float2(w0.y, w1.y), v2 = make_float2(w0.z, w1.z),
                 v3 = make_float2(w0.w, w1.w);
    float2 x0 = __bfloat1622float2(xr[0]), x1 = __bfloat1622float2(xr[1]), x2 = __bfloat1622float2(xr[2]);
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      const float2 x3 = __bfloat1622float2(xr[t + 3]);
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
  if (!full) {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (m0 + t < 0 || m0 + t >= s.len) y[t] = make_float2(0.f, 0.f);
  }
  if (!isq) {
#pragma unroll
    for (int t = 0; t < 32; ++t) {
      const float u = fabsf(y[t].x), v = fabsf(y[t].y);  // the finite ones
      mx = fmaxf(mx, fmaxf(u <= 3.4e38f ? u : 0.f, v <= 3.4e38f ? v : 0.f));
    }
  }
  const int R0 = (isq ? 0 : kC) + 32 * half;
#pragma unroll
  for (int t = 0; t < 32; ++t)
    tile_at<float2>(S.qk, sizeof(S.qk), f32_off(R0 + t, 2 * cp, 128 * 128)) =
        make_float2(umma::tf32_round(y[t].x), umma::tf32_round(y[t].y));
  umma::fence_proxy_async();
  umma::fence_before();
  __syncthreads();  // the tile written, S.kmax cleared
  umma::fence_after();
  const uint32_t tmem = S.tmem_base;
  if (tid == 0) {
    const uint64_t dq = umma::desc(smem_addr(S.qk), 16, 1024);
    constexpr uint32_t ID = umma::idesc_tf32(128, kC, false, false);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t ko = (k >> 2) * 16384 + (k & 3) * 32;
      umma::mma_tf32(tmem, umma::adv(dq, ko), umma::adv(dq, ko + 8192), ID, k > 0);
    }
    umma::commit(&S.bar);
  }
  if (!isq) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
    if (lane == 0) atomicMax(&S.kmax, m);
  }
  const bool late = !mbar_wait(&S.bar, 0);
  if (__syncthreads_or(late)) {  // also: S.kmax complete
    if (tid == 0) {
      report(p.err, GDN_DEV_ERR_TIMEOUT);
      mbar_wait(&S.bar, 0);
    }
  } else if (isq) {
    umma::fence_after();
    const int i = 32 * (warp & 3) + lane;
    float v[32];
    umma::tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 32 * half, v);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      tile_at<float4>(S.g, sizeof(S.g), g_off(i, 32 * half + 4 * q)) =
          make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  } else {
    const int e = scale_exp(S.kmax);
    const float f = exp2_int(e);
    // row r of a half's tile: in k's part of block (r >> 6), of block 2 + (r >> 6) for the low halves
    auto place = [](int r, int tok) {
      return (uint32_t)(r >> 6) * 16384u + 8192u + umma::sw128_off(r & 63, tok, 0);
    };
#pragma unroll
    for (int t8 = 0; t8 < 4; ++t8) {
      uint32_t h0[4], l0[4], h1[4], l1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = y[8 * t8 + 2 * i], v = y[8 * t8 + 2 * i + 1];
        split2(u.x * f, v.x * f, h0[i], l0[i]);
        split2(u.y * f, v.y * f, h1[i], l1[i]);
      }
      const uint32_t o0 = place(2 * cp, 32 * half + 8 * t8), o1 = place(2 * cp + 1, 32 * half + 8 * t8);
      tile_at<uint4>(S.qk, sizeof(S.qk), o0) = make_uint4(h0[0], h0[1], h0[2], h0[3]);
      tile_at<uint4>(S.qk, sizeof(S.qk), o0 + 32768) = make_uint4(l0[0], l0[1], l0[2], l0[3]);
      tile_at<uint4>(S.qk, sizeof(S.qk), o1) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
      tile_at<uint4>(S.qk, sizeof(S.qk), o1 + 32768) = make_uint4(l1[0], l1[1], l1[2], l1[3]);
    }
    if (tid == 64) GDN_GV(a.kscale, (long long)a.n_chunks * p.hk)[cslot * p.hk + hq] = exp2_int(-e);
  }
  umma::fence_proxy_async();
  umma::fence_before();
  __syncthreads();
  if (tid == 0) {
    const int64_t ri = cslot * p.hk + hq;
    if (GDN_SPAN_G(ri, 1, (long long)a.n_chunks * p.hk)) {
      Record& r = a.rec[ri];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        bulk_s2g(r.q + b * 8192, S.qk + b * 16384, 8192);
        bulk_s2g(r.kh + b * 8192, S.qk + b * 16384 + 8192, 8192);  // kh, then kl
      }
      bulk_s2g(r.g, S.g, kGBytes);
      bulk_commit();
      bulk_wait_all();
    }
  }
  if (warp == 0) umma::tmem_dealloc(tmem, 64);
}

// ---------------------------------------------------------------------------
// the chain
// ---------------------------------------------------------------------------
// Sixteen warps do the elementwise work; a seventeenth (the issuer, in a
// warpgroup of its own whose registers go to the others) issues every copy and
// product, because a thread that issues products is held up about as long as
// they run.  While the tensor core runs chunk c's products,
// the sixteen warps compute chunk c + 1's V (kept in registers) and P (the
// other of two buffers) and the gates of chunk c + 2; then they take chunk
// c's results and put chunk c + 1's operands in their place.
constexpr int kCompute = 512;
constexpr int kThreads = kCompute + 128;
// Registers per thread after the split of the launch's 640 x 96: the compute
// warps' state, V and temporaries against the issuer's few.
constexpr int kComputeRegs = 104, kIssuerRegs = 64;
static_assert(kCompute * kComputeRegs + 128 * kIssuerRegs <= kThreads * 96, "no more than the launch's registers");

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
  uint8_t pt[2][2 * NH * 64 * 128];  // P [head, i][j] tf32: two 32-column blocks
  uint8_t g[2][kGBytes];
  __nv_bfloat16 raw[2][kRawRows][128];
  __align__(128) __nv_bfloat16 ot[kC][128];
  // per chunk (mod 4) and head
  __align__(16) float b2[4][NH][kC];  // b log2(e)
  float eb[4][NH][kC];                // e^b
  float dt[4][NH][kC];
  float w[4][NH][kC];                 // e^{b_last - b} dt
  float dec[4][NH];                   // e^{b_last}
  uint32_t vmax[3];                   // largest |V w| of a chunk (mod 3), float bits
  uint32_t vfin;                      //   the same over finite values, where that is not finite
  uint64_t x_bar[2], g_bar[2], q_bar, k_bar, ready, o1_bar, mma_bar;
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
  // inconsistent, empty and padded sequences: ssm_check_kernel's
  if (!load_seq(p, n, s, bad_seq) || slot_class(s.slot, p.num_slots)) return;
  const int64_t seg_first = s.first / a.seg_chunks + n;
  const int seg = (int)(blockIdx.y - seg_first);
  const int n_seg = (s.nch + a.seg_chunks - 1) / a.seg_chunks;
  if (seg < 0 || seg >= n_seg || (STATE && seg == n_seg - 1)) return;
  const int c_begin = seg * a.seg_chunks, c_end = min(s.nch, c_begin + a.seg_chunks);
  const int nit = c_end - c_begin;
  const int64_t P0 = (s.p0 / kC + c_begin) * kC;  // the first chunk's first position

  if (warp == 0) umma::tmem_alloc(&S.tmem_base, TM_COLS);
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.x_bar[i], 1);
      mbar_init(&S.g_bar[i], 1);
    }
    mbar_init(&S.q_bar, 1);
    mbar_init(&S.k_bar, 1);
    mbar_init(&S.ready, kCompute / 32);
    mbar_init(&S.o1_bar, 1);
    mbar_init(&S.mma_bar, 1);
    S.vmax[0] = S.vmax[1] = S.vmax[2] = 0;
    fence_mbar_init();
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = S.tmem_base;
  constexpr uint32_t kPBlk = NH * 64 * 128;
  static_assert(TM_O1 == TM_S + kDK && TM_O2 == TM_O1 + kC && TM_V == TM_O2 + 2 * kC && TM_WH == TM_V + kC &&
                    TM_WL == TM_WH + kC / 2 && TM_WL + kC / 2 <= TM_COLS,
                "TMEM regions");

  if (warp >= kCompute / 32) {
    // ------------------------------------------------------------------ issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kIssuerRegs));
    if (warp == kCompute / 32) {
    constexpr uint32_t ID_O1 = umma::idesc_tf32(128, kC, false, false);
    constexpr uint32_t ID_O2 = umma::idesc_tf32(128, NH * kC, false, false);
    constexpr uint32_t ID_S = umma::idesc_f16(128, kDK, false, false);
    const int64_t rec0 = (s.first + c_begin) * p.hk + hq;
    auto bulk = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
      mbar_arrive_expect_tx(bar, bytes);
      if (GDN_GBYTES(src, bytes, a.rec, (long long)a.n_chunks * p.hk * sizeof(Record)) && GDN_SBYTES(dst, bytes, S))
        bulk_g2s(dst, src, bytes, bar);
    };
    // raw V rows and G of the segment's chunk i (lane 0)
    auto load_x = [&](int i) {
      const int32_t row0 = (int32_t)(s.t0 + (P0 + (int64_t)i * kC - 3 - s.p0));  // may be < 0: zeros
      mbar_arrive_expect_tx(&S.x_bar[i & 1], (uint32_t)sizeof(S.raw[0]));
      if (GDN_SPAN_G(2 * p.hk * kDK + tile * 128, 128, p.C) && GDN_SBYTES(&S.raw[i & 1][0][0], sizeof(S.raw[0]), S))
        tma_load_2d(&S.raw[i & 1][0][0], &xmap, 2 * p.hk * kDK + tile * 128, row0, &S.x_bar[i & 1]);
    };
    auto load_g = [&](int i) { bulk(S.g[i & 1], a.rec[rec0 + (int64_t)i * p.hk].g, kGBytes, &S.g_bar[i & 1]); };
    auto load_q = [&](int i) { bulk(S.q, a.rec[rec0 + (int64_t)i * p.hk].q, kQBytes, &S.q_bar); };
    auto load_k = [&](int i) { bulk(S.k, a.rec[rec0 + (int64_t)i * p.hk].kh, kKBytes, &S.k_bar); };
    int n_xg = 0, n_q = 0, n_k = 0, n_o1 = 0, n_mma = 0;  // issued
    if (lane == 0) {
      for (; n_xg < 2 && n_xg < nit; ++n_xg) {
        load_x(n_xg);
        if (!STATE) load_g(n_xg);
      }
      load_k(0);
      n_k = 1;
      if (!STATE) {
        load_q(0);
        n_q = 1;
      }
    }
    bool ok = true;
    const uint64_t dq = umma::desc(smem_addr(S.q), 16, 1024);
    const uint64_t dh = umma::desc(smem_addr(S.k), 16, 1024), dl = umma::adv(dh, sizeof(Record::kh));
    // pass i: chunk i's operands are in place (and chunk i - 1's output staged)
    for (int i = 0; i < nit + (STATE ? 0 : 1) && ok; ++i) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&S.ready, i & 1)))) break;
      umma::fence_after();
      const uint32_t par = i & 1;
      if (lane == 0 && i < nit) {
        if (i + 2 < nit) {  // chunk i's raw rows and G have been read
          load_x(i + 2);
          if (!STATE) load_g(i + 2);
          n_xg = i + 3;
        }
        if (!STATE) {
          // O1^T = S^T Q^T
          if ((ok = mbar_wait(&S.q_bar, par))) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              umma::mma_tf32_ta(tmem + TM_O1, tmem + TM_S + 8 * k, umma::adv(dq, (k >> 2) * 8192 + (k & 3) * 32),
                                ID_O1, k > 0);
            umma::commit(&S.o1_bar);
            ++n_o1;
          }
        }
      }
      if constexpr (!STATE) {
        // chunk i - 1's staged output
        if (i > 0) {
          const int64_t P = P0 + (int64_t)(i - 1) * kC;
          const int tlo = (int)max((int64_t)0, s.p0 - P), thi = (int)min((int64_t)kC, s.p1 - P);
          if (tlo == 0 && thi == kC) {
            if (lane == 0 && GDN_SPAN_G(s.t0 + (P - s.p0), kC, p.total)) {
              tma_store_2d(&omap, &S.ot[0][0], tile * 128, (int32_t)(s.t0 + (P - s.p0)));
              bulk_commit();
            }
          } else {
            const auto ot = GDN_SV(&S.ot[0][0], kC * 128);
            const auto out = GDN_GV(reinterpret_cast<__nv_bfloat16*>(p.out), p.total * p.hv * DV);
            for (int r = tlo + (lane >> 4); r < thi; r += 2)
              vec_at<uint4>(out, ((s.t0 + P - s.p0 + r) * p.hv) * DV + tile * 128 + 8 * (lane & 15)) =
                  vec_at<const uint4>(ot, r * 128 + 8 * (lane & 15));
            __syncwarp();
          }
        }
      }
      if (lane == 0 && i < nit && ok) {
        if (!STATE) {
          // O2^T = V^T P^T
          const uint64_t dp = umma::desc(smem_addr(S.pt[par]), 16, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma::mma_tf32_ta(tmem + TM_O2, tmem + TM_V + 8 * k, umma::adv(dp, (k >> 2) * kPBlk + (k & 3) * 32),
                              ID_O2, k > 0);
          // dS^T takes the place of S^T once O1's product has read it
          if ((ok = mbar_wait(&S.o1_bar, par)) && i + 1 < nit) {
            load_q(i + 1);
            ++n_q;
          }
        }
        if (ok && (ok = mbar_wait(&S.k_bar, par))) {
          umma::fence_after();
          // dS^T = (V w)^T K, small products first
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ta(tmem + TM_S, tmem + TM_WL + 8 * k, umma::adv(dh, 32 * k), ID_S, k > 0);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ta(tmem + TM_S, tmem + TM_WH + 8 * k, umma::adv(dl, 32 * k), ID_S, true);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ta(tmem + TM_S, tmem + TM_WH + 8 * k, umma::adv(dh, 32 * k), ID_S, true);
          bulk_wait_read();  // the staging may be written once this chunk's products are known to be done
          umma::commit(&S.mma_bar);
          ++n_mma;
          if ((ok = mbar_wait(&S.mma_bar, par)) && i + 1 < nit) {
            load_k(i + 1);
            ++n_k;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (!ok) {
        // a wait expired: let what is in flight land before the memory goes
        report(p.err, GDN_DEV_ERR_TIMEOUT);
        for (int k = max(0, n_xg - 2); k < n_xg; ++k) {
          mbar_wait(&S.x_bar[k & 1], (k >> 1) & 1);
          if (!STATE) mbar_wait(&S.g_bar[k & 1], (k >> 1) & 1);
        }
        if (n_q) mbar_wait(&S.q_bar, (n_q - 1) & 1);
        if (n_k) mbar_wait(&S.k_bar, (n_k - 1) & 1);
        if (n_o1) mbar_wait(&S.o1_bar, (n_o1 - 1) & 1);
        if (n_mma) mbar_wait(&S.mma_bar, (n_mma - 1) & 1);
      }
      bulk_wait_all();
    }
    }
  } else {
    // ----------------------------------------------------------------- compute
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kComputeRegs));
    const int lrow = 32 * (warp & 3) + lane;  // V channel of the tile, TMEM lane
    const int qq = warp >> 2;                 // token (or dk column) quarter
    const int hl = lrow / DV;                 // this row's head within the tile
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int ch = 2 * p.hk * kDK + tile * 128 + lrow;

    // gates: warps 8 and 10, which have no part in P; two tokens per lane,
    // their logits loaded one chunk ahead
    const bool gate_warp = warp == 8 || (NH == 2 && warp == 10);
    const int gh = h0 + (warp == 10 ? NH - 1 : 0), ghl = gh - h0;
    const auto gate_a = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.a), p.total * p.hv);
    float ga[2] = {0.f, 0.f};
    auto gate_load = [&](int i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t m = P0 + (int64_t)i * kC + 32 * e + lane - s.p0;
        ga[e] = i < nit && m >= 0 && m < s.len ? __bfloat162float(gate_a[(s.t0 + m) * p.hv + gh]) : 0.f;
      }
    };
    const float A_log = GDN_GV(p.A_log, p.hv)[gh], dtb = GDN_GV(p.dt_bias, p.hv)[gh];
    auto gates = [&](int i) {
      const int buf = i & 3;
      float dt[2], b[2], suf[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t m = P0 + (int64_t)i * kC + 32 * e + lane - s.p0;
        const bool in = m >= 0 && m < s.len;
        const Gate t = gate(A_log, dtb, ga[e]);
        dt[e] = in ? t.dt : 0.f;
        b[e] = suf[e] = in ? floor_log_decay(t.g) : 0.f;
      }
      gate_load(i + 1);
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
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 32 * e + lane;
        S.b2[buf][ghl][t] = b[e] * 1.4426950408889634f;
        S.eb[buf][ghl][t] = expf(b[e]);
        S.dt[buf][ghl][t] = dt[e];
        S.w[buf][ghl][t] = expf(suf[e]) * dt[e];
      }
      if (lane == 0) S.dec[buf][ghl] = expf(all);
    };
    if (gate_warp) {
      gate_load(0);
      gates(0);
      if (nit > 1) gates(1);
    }

    // the state entering the segment, S^T row lrow, columns 32 qq ..
    float st[32];
    float seg_dec = 1.f;
    const size_t tile_off = ((size_t)tile * 128 + lrow) * kDK + 32 * qq;  // within one slot's [hv][dv][dk]
    const long long slot_n = (long long)p.hv * DV * kDK;
    const auto segs = GDN_GV(a.seg_state, a.n_segs * slot_n);
    const auto pool = GDN_GV(p.ssm, p.num_slots * slot_n) + ((size_t)s.slot * slot_n + tile_off);
    {
      // One segment: from the slot.  Several: the first launch starts the
      // first segment from the slot and keeps a copy, at the last segment's
      // otherwise unused place, for the second launch; the others from zero.
      const auto keep = segs + (n_seg > 1 ? (seg_first + n_seg - 1) * slot_n + (int64_t)tile_off : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (seg == 0) {
          v = STATE || n_seg == 1 ? vec_at<const float4>(pool, 4 * i) : vec_at<const float4>(keep, 4 * i);
          if (STATE) vec_at<float4>(keep, 4 * i) = v;
        }
        st[4 * i] = v.x; st[4 * i + 1] = v.y; st[4 * i + 2] = v.z; st[4 * i + 3] = v.w;
      }
      if (!STATE) {
        for (int k = 0; k < seg; ++k) {
          const auto L = segs + ((seg_first + k) * slot_n + (int64_t)tile_off);
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
    const float4 w4 = vec_at<const float4>(GDN_GV(p.conv_w, (long long)p.C * 4), (size_t)ch * 4);
    const float bias = p.conv_bias ? GDN_GV(p.conv_bias, p.C)[ch] : 0.f;
    // P's rows of this thread: row pr of the heads' 64 NH, PC columns from pc;
    // what lies above the diagonal stays zero
    constexpr int PC = 8 * NH;
    const int pr = NH == 2 ? lrow : (lrow & 63), pi = pr & 63, ph = pr >> 6;
    const int pc = 16 * qq + (NH == 2 ? 0 : 8 * (lrow >> 6));
    const float skip = p.D ? GDN_GV(p.D, p.hv)[h0 + ph] : 0.f;
    if (!STATE) {
#pragma unroll
      for (int c4 = 0; c4 < PC / 4; ++c4) {
        tile_at<float4>(S.pt[0], sizeof(S.pt[0]), f32_off(pr, pc + 4 * c4, kPBlk)) = make_float4(0.f, 0.f, 0.f, 0.f);
        tile_at<float4>(S.pt[1], sizeof(S.pt[1]), f32_off(pr, pc + 4 * c4, kPBlk)) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    const int kpc = p.ckpt_block / kC;
    const int q0 = (int)((s.p0 / kC) % kpc);
    auto ckpt_slot = [&](int c) -> int32_t {  // checkpoint slot at the end of the sequence's chunk c, -1: none
      if (c == s.nch - 1 && s.p1 % kC) return -1;
      const int q = q0 + c + 1;
      if (q % kpc) return -1;
      const int idx = q / kpc - 1;
      if (idx >= p.max_ckpt) return -1;
      const int32_t id = GDN_GV(p.ckpt_ids, (long long)p.n_seq * p.max_ckpt)[(size_t)n * p.max_ckpt + idx];
      return slot_class(id, p.ck_num_slots) == 0 ? id : -1;
    };

    bool bad = false;
    float y[16];  // V of the next chunk: channel lrow, tokens 16 qq ..
    auto weights = [&](int i, float (&x)[16]) {  // V w
      const auto ws = GDN_SV(&S.w[i & 3][hl][0], kC);
#pragma unroll
      for (int t4 = 0; t4 < 4; ++t4) {
        const float4 v = vec_at<const float4>(ws, 16 * qq + 4 * t4);
        x[4 * t4] = y[4 * t4] * v.x;
        x[4 * t4 + 1] = y[4 * t4 + 1] * v.y;
        x[4 * t4 + 2] = y[4 * t4 + 2] * v.z;
        x[4 * t4 + 3] = y[4 * t4 + 3] * v.w;
      }
    };
    // V and P of the segment's chunk i, the largest |V w|, the gates ahead
    auto features = [&](int i) {
      const int64_t P = P0 + (int64_t)i * kC;
      if (!mbar_wait(&S.x_bar[i & 1], (i >> 1) & 1)) bad = true;
      if (P - 3 < s.p0) {
        // the up to 3 rows just before the sequence come from the history
        const int64_t lo = max(P - 3, s.p0 - 3), hi = min(P + kC, s.p0);
        const auto hist = GDN_GV(reinterpret_cast<const __nv_bfloat16*>(p.conv), (long long)p.num_slots * 3 * p.C) +
                          (size_t)s.slot * 3 * p.C;
        for (int64_t pos = lo; pos < hi; ++pos)
          if (tid < 128)
            S.raw[i & 1][GDN_S((int)(pos - (P - 3)), kRawRows)][tid] =
                hist[(size_t)(3 - (s.p0 - pos)) * p.C + 2 * p.hk * kDK + tile * 128 + tid];
        umma::fence_proxy_async();  // before a later chunk's copy into these rows
        named_sync(1, kCompute);
      }
      {
        const auto xs = GDN_SV(&S.raw[i & 1][0][0], kRawRows * 128) + (16 * qq * 128 + lrow);
        float x[19];
#pragma unroll
        for (int r = 0; r < 19; ++r) x[r] = __bfloat162float(xs[r * 128]);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          float acc = fmaf(w4.x, x[t], bias);
          acc = fmaf(w4.y, x[t + 1], acc);
          acc = fmaf(w4.z, x[t + 2], acc);
          acc = fmaf(w4.w, x[t + 3], acc);
          y[t] = silu_acc(acc);
        }
      }
      if (P < s.p0 || P + kC > s.p1) {  // tokens outside the sequence
        const int tlo = (int)max((int64_t)0, s.p0 - P), thi = (int)min((int64_t)kC, s.p1 - P);
#pragma unroll
        for (int t = 0; t < 16; ++t)
          if (16 * qq + t < tlo || 16 * qq + t >= thi) y[t] = 0.f;
      }
      {
        float x[16];
        weights(i, x);
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < 16; ++t) m = max(m, __float_as_uint(x[t]) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) atomicMax(&S.vmax[i % 3], m);
      }
      if constexpr (!STATE) {
        if (!mbar_wait(&S.g_bar[i & 1], (i >> 1) & 1)) bad = true;
        if (pc <= pi) {
          const int buf = i & 3;
          const float bi = S.b2[buf][ph][pi];
#pragma unroll
          for (int c4 = 0; c4 < PC / 4; ++c4) {
            const int j = pc + 4 * c4;
            const float4 gv = tile_at<float4>(S.g[i & 1], sizeof(S.g[0]), g_off(pi, j));
            const float4 bj = *reinterpret_cast<const float4*>(&S.b2[buf][ph][GDN_S(j, kC - 3)]);
            const float4 dj = *reinterpret_cast<const float4*>(&S.dt[buf][ph][j]);
            float e[4] = {bi - bj.x, bi - bj.y, bi - bj.z, bi - bj.w};
            const float gd[4] = {gv.x * dj.x, gv.y * dj.y, gv.z * dj.z, gv.w * dj.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x;
              asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(x) : "f"(e[k]));
              x *= gd[k];
              if (j + k == pi) x += skip;
              e[k] = j + k <= pi ? umma::tf32_round(x) : 0.f;
            }
            tile_at<float4>(S.pt[i & 1], sizeof(S.pt[0]), f32_off(pr, j, kPBlk)) = make_float4(e[0], e[1], e[2], e[3]);
          }
        }
      }
      if (gate_warp && i + 1 < nit && i > 0) gates(i + 1);
      if (tid == 0) S.vmax[(i + 1) % 3] = 0;
    };
    int ve = 0;  // scale exponent of the (V w) operand in TMEM
    // chunk i's operands into TMEM (its vmax complete): S^T, V^T, (V w)^T
    auto operands = [&](int i) {
      if constexpr (!STATE) {
        float r[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = umma::tf32_round(st[e]);
        umma::tmem_st32(tlane + TM_S + 32 * qq, r);
        float v[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) v[t] = umma::tf32_round(y[t]);
        umma::tmem_st16(tlane + TM_V + 16 * qq, v);
      }
      float x[16];
      weights(i, x);
      uint32_t m = S.vmax[i % 3];
      if (m >= 0x7f800000u) {
        // infinite or NaN values among V w: the scale of the finite ones
        named_sync(1, kCompute);
        if (tid == 0) S.vfin = 0;
        named_sync(1, kCompute);
        m = 0;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const uint32_t u = __float_as_uint(x[t]) & 0x7fffffffu;
          m = max(m, u < 0x7f800000u ? u : 0u);
        }
        atomicMax(&S.vfin, m);
        named_sync(1, kCompute);
        m = S.vfin;
      }
      ve = scale_exp(m);
      const float f = exp2_int(ve);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) split2(x[2 * t] * f, x[2 * t + 1] * f, hi[t], lo[t]);
      __syncwarp();
      tmem_st8(tlane + TM_WH + 8 * qq, hi);
      tmem_st8(tlane + TM_WL + 8 * qq, lo);
    };
    auto publish = [&]() {
      umma::fence_proxy_async();
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.ready);
    };

    named_sync(1, kCompute);  // the first gates
    features(0);
    int i = 0;
    if (!named_sync_or(1, kCompute, bad)) {
      operands(0);
      publish();
      for (; i < nit; ++i) {
        if (i + 1 < nit) features(i + 1);
        const float kscale = GDN_GV(a.kscale, (long long)a.n_chunks * p.hk)[(s.first + c_begin + i) * p.hk + hq];
        if (named_sync_or(1, kCompute, bad)) break;
        if (!mbar_wait(&S.mma_bar, i & 1)) bad = true;
        __syncwarp();
        umma::fence_after();
        const int buf = i & 3;
        {
          const float dec = S.dec[buf][hl], f = exp2_int(-ve);
          seg_dec *= dec;
          float d[32];
          umma::tmem_ld32(tlane + TM_S + 32 * qq, d);
#pragma unroll
          for (int e = 0; e < 32; ++e) st[e] = fmaf(st[e], dec, d[e] * kscale * f);
        }
        if constexpr (!STATE) {
          float o1[16], o2[16];
          umma::tmem_ld16(tlane + TM_O1 + 16 * qq, o1);
          umma::tmem_ld16(tlane + TM_O2 + (NH == 2 ? hl * kC : 0) + 16 * qq, o2);
          const auto ot = GDN_SV(&S.ot[0][0], kC * 128);
#pragma unroll
          for (int t4 = 0; t4 < 4; ++t4) {
            const float4 e = *reinterpret_cast<const float4*>(&S.eb[buf][hl][GDN_S(16 * qq + 4 * t4, kC - 3)]);
            const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ot[(16 * qq + 4 * t4 + k) * 128 + lrow] = __float2bfloat16_rn(fmaf(o1[4 * t4 + k], ev[k], o2[4 * t4 + k]));
          }
          const int32_t cid = ckpt_slot(c_begin + i);
          if (cid >= 0) {
            const auto K = GDN_GV(p.ck_ssm, p.ck_num_slots * slot_n) + ((size_t)cid * slot_n + tile_off);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              vec_at<float4>(K, 4 * e) = make_float4(st[4 * e], st[4 * e + 1], st[4 * e + 2], st[4 * e + 3]);
          }
        }
        if (i + 1 < nit) operands(i + 1);
        if (i + 1 < nit || !STATE) publish();
      }
    }
    bad = named_sync_or(1, kCompute, bad);
    if (i == nit && !bad) {
      if (STATE) {
        const auto L = segs + ((seg_first + seg) * slot_n + (int64_t)tile_off);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          vec_at<float4>(L, 4 * e) = make_float4(st[4 * e], st[4 * e + 1], st[4 * e + 2], st[4 * e + 3]);
        if (qq == 0 && lrow % DV == 0)
          GDN_GV(a.seg_decay, (long long)a.n_segs * p.hv)[(seg_first + seg) * p.hv + h0 + hl] = seg_dec;
      } else if (seg == n_seg - 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          vec_at<float4>(pool, 4 * e) = make_float4(st[4 * e], st[4 * e + 1], st[4 * e + 2], st[4 * e + 3]);
      }
    } else if (tid == 0) {
      report(p.err, GDN_DEV_ERR_TIMEOUT);
    }
  }
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
