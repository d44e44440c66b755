// Chunked prefill of linear attention with a fixed decay on the 5th-generation
// tensor cores (dk = dv = 128, bf16 activations).
//
// The published chunk form, in chunks of 64 tokens aligned to absolute
// positions (shorter at both ends of a sequence).  Token t of a chunk of L,
// t = 0 .. L - 1, of one V head:
//   O_t = scale (sum_{j <= t} lambda^(t - j) (q_t . k_j) v_j + lambda^(t + 1) S^T q_t)
//   S  <- lambda^L S + sum_j lambda^(L - 1 - j) k_j v_j^T
// One CTA per (V head, sequence or segment of one) walks its chunks in order,
// V channels in the tensor core's M = 128 rows, with S^T [dv][dk] in registers
// in fp32 between chunks.  Per chunk, all accumulators in TMEM:
//   G    = Q K^T                    Q and K as they lie in memory
//   dS^T = (V w)^T K                w_j = lambda^(L - 1 - j); A = V w, in parts
//   O1^T = S^T Q^T                  A = S^T in TMEM, two parts
//   O2^T = V^T P^T                  A = V; B = P, its two parts side by side
// dS does not need S, so only an elementwise update per chunk is left of the
// recurrence, and the tensor core always has another chunk's work.
//
// Roundings.  q, k and v are bf16 already and enter G, dS and O2 exactly.
// V w is split into three bf16 parts (24 bits: the fp32 product itself), so that
// states keep fp32's accuracy; P and S^T, which only outputs see, into two (16
// bits, off by at most 2^-17 of each term, against the output's own 2^-9).
// Parts of 8 bits keep fp32's range, so no scaling is needed; values from
// 3.39e38 on become infinite.
//
// 20 warps by role: 8 hold S (2 per 32 V channels, 64 dk columns each), 4 write
// outputs, 3 compute P (in blocks of 32 x 32; one of four lies above the
// diagonal), 4 scale and split V, one issues the products.
#include "lin.cuh"

#include "decode_tma.cuh"  // sm_count
#include "ssm.cuh"         // allow_smem
#include "tma.cuh"
#include "umma.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kD = 128;  // dk = dv
constexpr int kStages = 3;
constexpr int kStateWarps = 8, kOutWarp = 8, kAuxWarp = 12, kIssuer = 16;
constexpr int kThreads = 20 * 32;
constexpr int kStateThreads = kStateWarps * 32;
// Registers per thread, by warpgroup; 640 x 96 at launch is what there is.
constexpr int kStateRegs = 136, kOutRegs = 72, kAuxRegs = 64;
static_assert(2 * kStateRegs + kOutRegs + 2 * kAuxRegs <= 5 * 96, "the launch's registers");

// TMEM columns
constexpr uint32_t TM_G = 0, TM_DS = 64, TM_O1 = 192, TM_O2 = 256, TM_SH = 384, TM_SL = 448, TM_COLS = 512;

struct __align__(1024) Stage {
  uint8_t qk[2][128 * 128];  // 64-column blocks: rows 0..63 q, 64..127 k
  uint8_t v[2][64 * 128];    // 64-column blocks
};
struct __align__(1024) ChunkSmem {
  Stage st[kStages];
  uint8_t vw[3][2 * 64 * 128];  // V w: its three parts
  uint8_t p[2][128 * 128];      // P [t][j] by the chunk's parity: rows 0..63 hi, 64..127 lo
  float pw[kC + 1];             // lambda^n
  float ps[kC + 1];             // scale lambda^n
  Segment seg;
  int some;
  uint64_t full[kStages], empty[kStages];
  uint64_t g_full, aux_full, ds_full, ds_empty, s_full, o_full, o_empty, init, drained;
  uint32_t tmem_base;
};
// The state tile's way between global memory and the threads' rows: 64 KB from
// the last stage on, free before chunk kStages - 1 is loaded and V w first
// written, and after the last product.
constexpr unsigned kTile = kD * kD * 4;
static_assert(sizeof(ChunkSmem) + 1024 <= 232448, "shared memory of a CTA");
static_assert(offsetof(ChunkSmem, p) - offsetof(ChunkSmem, st) - (kStages - 1) * sizeof(Stage) >= kTile, "state tile");

// hi: x rounded to bf16, packed in pairs; x: what is left of it, exactly
__device__ __forceinline__ uint32_t take_bf16(float2& x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  const uint32_t hi = *reinterpret_cast<const uint32_t*>(&h);
  x = fma2(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), make_float2(-1.f, -1.f), x);
  return hi;
}
// x as two bf16 parts, packed in pairs
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = take_bf16(x);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x.x, x.y);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// 16 TMEM columns of packed values, written; complete after tmem_wait_st()
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&v)[16], int line = __builtin_LINE()) {
  if (!umma::tmem_ok(taddr, 16, true, line)) return;
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// three runs of 8 columns read at once
__device__ __forceinline__ void tmem_ld8x3(uint32_t ta, uint32_t tb, uint32_t tc, float (&va)[8], float (&vb)[8],
                                           float (&vc)[8], int line = __builtin_LINE()) {
  if (!umma::tmem_ok(ta, 8, true, line) || !umma::tmem_ok(tb, 8, true, line) || !umma::tmem_ok(tc, 8, true, line)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) va[i] = vb[i] = vc[i] = 0.f;
    return;
  }
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(va[0]), "=f"(va[1]), "=f"(va[2]), "=f"(va[3]), "=f"(va[4]), "=f"(va[5]), "=f"(va[6]), "=f"(va[7]),
        "=f"(vb[0]), "=f"(vb[1]), "=f"(vb[2]), "=f"(vb[3]), "=f"(vb[4]), "=f"(vb[5]), "=f"(vb[6]), "=f"(vb[7]),
        "=f"(vc[0]), "=f"(vc[1]), "=f"(vc[2]), "=f"(vc[3]), "=f"(vc[4]), "=f"(vc[5]), "=f"(vc[6]), "=f"(vc[7])
      : "r"(ta), "r"(tb), "r"(tc)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Products issued by a whole converged warp, of which the thread with `lead`
// set does it: descriptors and addresses that are the same for the warp stay in
// its uniform registers, where the instruction wants them.  (Issued by one
// thread alone, each product took some 100 cycles to assemble.)
// D (TMEM) (+)= A B, both by descriptor
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate, int line = __builtin_LINE()) {
  if (!umma::tmem_ok(tmem_d, umma::idesc_n(idesc), false, line)) return;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
      : "memory");
}
// the same with A in TMEM (K = 16 values in 8 columns)
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc,
                                       bool accumulate, int line = __builtin_LINE()) {
  if (!umma::tmem_ok(tmem_d, umma::idesc_n(idesc), false, line) || !umma::tmem_ok(tmem_a, 8, false, line)) return;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(bar)),
      "r"(lead)
      : "memory");
}

__device__ __forceinline__ void st_global32(float* to, float4 a, float4 b) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to), "f"(a.x), "f"(a.y), "f"(a.z), "f"(a.w),
               "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
               : "memory");
}

// wait of a whole warp
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// grid (V heads, segment slots).  STATE: the segment's own state alone (every
// segment but a sequence's last).
template <bool STATE>
__global__ void __launch_bounds__(kThreads, 1)
    lin_chunk_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChunkSmem& S = *reinterpret_cast<ChunkSmem*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one value per warp
  const int h = blockIdx.x, hq = h / a.G;
  if (warp == 1) umma::tmem_alloc(&S.tmem_base, TM_COLS);
  if (tid == 64) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.g_full, 1);
    mbar_init(&S.aux_full, STATE ? 4 : 4 + 3);
    mbar_init(&S.ds_full, 1);
    mbar_init(&S.ds_empty, kStateWarps);
    mbar_init(&S.s_full, kStateWarps);
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_empty, 4);
    mbar_init(&S.init, kStateWarps);
    mbar_init(&S.drained, 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    Segment s;
    const bool some = find_segment(a, blockIdx.y, s, !STATE && lane == 0 && h == 0);
    if (lane == 0) {
      S.seg = s;
      S.some = some && !(STATE && (s.seg == s.n_seg - 1 || s.padded));
    }
  }
  if (tid >= 96 && tid < 96 + kC + 1) {
    const int n = tid - 96;
    const float p = power(GDN_GV(a.log_decay, a.hv)[h], n);
    S.pw[n] = p;
    S.ps[n] = p * a.scale;
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = S.tmem_base;
  const int64_t ld = (int64_t)a.hv * kD;
  if (!S.some || S.seg.padded) {
    if (S.some) {  // outputs of an unusable slot: zeros
      const auto out = GDN_GV(reinterpret_cast<uint4*>(a.out), a.total * ld / 8);
      const int64_t n = (S.seg.m1 - S.seg.m0) * (kD / 8);
      for (int64_t e = tid; e < n; e += kThreads)
        out[((S.seg.t0 + S.seg.m0 + e / (kD / 8)) * ld + (int64_t)h * kD) / 8 + e % (kD / 8)] = make_uint4(0, 0, 0, 0);
    }
    if (warp == 1) umma::tmem_dealloc(tmem, TM_COLS);
    return;
  }
  // chunk i holds the segment's tokens [from(i), from(i) + count(i))
  const int64_t m0 = S.seg.m0, m1 = S.seg.m1;
  const int head = (int)((S.seg.p0 + m0) % kC);  // 0 but for a sequence's first chunk
  const int nit = (int)((m1 - m0 + head + kC - 1) / kC);
  auto from = [&](int i) { return i ? m0 - head + (int64_t)i * kC : m0; };
  auto count = [&](int i) { return (int)(min(m1, m0 - head + (int64_t)(i + 1) * kC) - from(i)); };

  if (warp >= kAuxWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kAuxRegs));
    const int quarter = warp & 3, half = (warp - kAuxWarp) >> 2;
    if (warp == kIssuer) {
      // ---------------------------------------------------------------- issuer
      // Order per chunk i: dS(i), G(i + 1), O2(i), O1(i): whatever the other
      // warps make of one product has two more products' time.
      constexpr uint32_t ID_64 = umma::idesc_bf16(128, kC, false, false);  // G, O1
      constexpr uint32_t ID_DS = umma::idesc_bf16(128, kD, true, true);
      constexpr uint32_t ID_O2 = umma::idesc_bf16(128, 2 * kC, true, false);
      const uint32_t lead = lane == 0;
      const uint64_t dq0 = umma::desc(smem_addr(S.st[0].qk[0]), 16, 1024);            // q as rows, k 8 KB on
      const uint64_t dk0 = umma::desc(smem_addr(S.st[0].qk[0]) + 8192, 16384, 1024);  // k as columns
      const uint64_t dv0 = umma::desc(smem_addr(S.st[0].v[0]), 8192, 1024);
      const uint64_t dvw = umma::desc(smem_addr(S.vw[0]), 8192, 1024);
      const uint64_t dp0 = umma::desc(smem_addr(S.p[0]), 16, 1024);
      bool ok = true;
      auto issue_g = [&](int s) {
        const uint64_t d = umma::adv(dq0, s * (uint32_t)sizeof(Stage));
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
          mma_ss(lead, tmem + TM_G, umma::adv(d, at), umma::adv(d, 8192 + at), ID_64, k > 0);
        }
        commit(lead, &S.g_full);
      };
      if ((ok = wait_all(&S.full[0], 0)) && !STATE) {
        umma::fence_after();
        issue_g(0);
      }
      int s = 0, s_par = 0;  // chunk i's stage and its phase
#pragma unroll 1
      for (int i = 0; i < nit && ok; ++i) {
        const uint32_t at = s * (uint32_t)sizeof(Stage);
        const int s1 = s + 1 == kStages ? 0 : s + 1, s1_par = s1 ? s_par : s_par ^ 1;
        // dS^T = (V w)^T K, the small parts first.  V w and P of this chunk are
        // there (so G's columns have been read, too).
        ok = wait_all(&S.aux_full, i & 1) && (i == 0 || wait_all(&S.ds_empty, (i - 1) & 1));
        if (!ok) break;
        umma::fence_after();
        {
          const uint64_t dk = umma::adv(dk0, at);
#pragma unroll
          for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(lead, tmem + TM_DS, umma::adv(dvw, part * 16384 + 2048 * k), umma::adv(dk, 2048 * k), ID_DS,
                     part < 2 || k > 0);
          commit(lead, &S.ds_full);
          if (STATE) commit(lead, &S.empty[s]);
        }
        if (i + 1 < nit) {
          if (!(ok = wait_all(&S.full[s1], s1_par))) break;
          if (!STATE) {
            umma::fence_after();
            issue_g(s1);
          }
        }
        if (!STATE) {
          // O2^T = V^T P^T, both parts of P side by side
          if (i > 0 && !(ok = wait_all(&S.o_empty, (i - 1) & 1))) break;
          umma::fence_after();
          {
            const uint64_t dv = umma::adv(dv0, at), dp = umma::adv(dp0, (i & 1) * (uint32_t)sizeof(S.p[0]));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(lead, tmem + TM_O2, umma::adv(dv, 2048 * k), umma::adv(dp, 32 * k), ID_O2, k > 0);
          }
          // O1^T = S^T Q^T
          if (!(ok = wait_all(&S.s_full, i & 1))) break;
          umma::fence_after();
          {
            const uint64_t dq = umma::adv(dq0, at);
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_ts(lead, tmem + TM_O1, tmem + (part ? TM_SL : TM_SH) + 8 * k,
                       umma::adv(dq, (k >> 2) * 16384 + (k & 3) * 32), ID_64, part == 0 || k > 0);
            commit(lead, &S.o_full);
          }
        }
        s = s1;
        s_par = s1_par;
      }
      if (!ok && lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
      // the products in flight end before their memory is used otherwise
      commit(lead, &S.drained);
      wait_all(&S.drained, 0);
    } else if (quarter >= 2) {
      // ------------------------------------------------------------- V w, split
      // A thread has 8 of the tile's 1024 16-byte pieces, of four rows.
      const int ct = ((quarter - 2) * 2 + half) * 32 + lane;  // 0 .. 127
      bool ok = wait_all(&S.init, 0);                         // the state tile has left vw
      for (int i = 0; i < nit && ok; ++i) {
        Stage& st = S.st[i % kStages];
        const int L = count(i);
        if (!(ok = wait_all(&S.full[i % kStages], (i / kStages) & 1))) break;
        if (L < kC) {
          // rows behind the chunk are others' values: zeros, or a NaN among
          // them would reach this chunk's products
#pragma unroll 1
          for (int e = ct; e < (kC - L) * 8; e += 128) {
            const uint32_t at = (uint32_t)(L + e / 8) * 128u + (e % 8) * 16u;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              tile_at<uint4>(st.v[b], sizeof(st.v[b]), at) = make_uint4(0, 0, 0, 0);
              tile_at<uint4>(st.qk[b], sizeof(st.qk[b]), 8192 + at) = make_uint4(0, 0, 0, 0);
            }
          }
          umma::fence_proxy_async();
          named_sync(2, 128);
        }
        if (i > 0 && !(ok = wait_all(&S.ds_full, (i - 1) & 1))) break;  // vw was read
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int row = (e & 3) * 16 + ct / 8;
          const uint32_t at = (uint32_t)row * 128u + (ct & 7) * 16u;
          const float w = row < L ? S.pw[L - 1 - row] : 0.f;
          const uint4 u = tile_at<const uint4>(st.v[e >> 2], sizeof(st.v[0]), at);
          const uint32_t x[4] = {u.x, u.y, u.z, u.w};
          uint32_t r[3][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 y = mul2(make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u)),
                            make_float2(w, w));
            r[0][k] = take_bf16(y);
            r[1][k] = take_bf16(y);
            const __nv_bfloat162 l = __floats2bfloat162_rn(y.x, y.y);
            r[2][k] = *reinterpret_cast<const uint32_t*>(&l);
          }
#pragma unroll
          for (int q = 0; q < 3; ++q)
            tile_at<uint4>(S.vw[q], sizeof(S.vw[0]), (e >> 2) * 8192u + at) = make_uint4(r[q][0], r[q][1], r[q][2], r[q][3]);
        }
        umma::fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.aux_full);
      }
      if (!ok && lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
    } else if (!STATE) {
      // ---------------------------------------------------------------------- P
      // token row t, columns 32 half .. + 31
      const int t = 32 * quarter + lane, j0 = 32 * half;
      const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);
      if (quarter == 0) {  // the block above the diagonal: zeros, once
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t at = umma::sw128_off(t, 32 + 8 * c, 0);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            tile_at<uint4>(S.p[b], sizeof(S.p[0]), at) = make_uint4(0, 0, 0, 0);
            tile_at<uint4>(S.p[b], sizeof(S.p[0]), 8192 + at) = make_uint4(0, 0, 0, 0);
          }
        }
      }
      bool ok = true;
      for (int i = 0; i < nit && ok; ++i) {
        if (!(ok = wait_all(&S.g_full, i & 1))) break;
        umma::fence_after();
        // G(i)'s commit covers the products before it, O2(i - 2) among them: P's
        // buffer is free
        uint8_t* const pt = S.p[i & 1];
        {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float g[16];
            umma::tmem_ld16(tlane + TM_G + j0 + 16 * q, g);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = 8 * c + 2 * k;
                const int d = t - j0 - 16 * q - e;  // t - j
                split2(make_float2(d >= 0 ? g[e] * S.ps[max(d, 0)] : 0.f, d >= 1 ? g[e + 1] * S.ps[max(d - 1, 0)] : 0.f),
                       hi[k], lo[k]);
              }
              const uint32_t at = umma::sw128_off(t, j0 + 16 * q + 8 * c, 0);
              tile_at<uint4>(pt, sizeof(S.p[0]), at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              tile_at<uint4>(pt, sizeof(S.p[0]), 8192 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
          umma::fence_proxy_async();
        }
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.aux_full);
      }
      if (!ok && lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
    }
  } else if (warp >= kOutWarp) {
    // ------------------------------------------------------------------ outputs
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOutRegs));
    // Warp kOutWarp also issues the copies: chunk i + kStages once chunk i's
    // products are done (and its V split, which dS waited for).
    const int64_t kd = (int64_t)a.hk * kD;
    const bool loader = warp == kOutWarp;
    int n_load = 0;
    auto load = [&]() {  // chunk n_load
      const int s = n_load % kStages;
      if (lane == 0) {
        Stage& st = S.st[s];
        const int32_t row = (int32_t)(S.seg.t0 + from(n_load));
        mbar_arrive_expect_tx(&S.full[s], (STATE ? 4 : 6) * 8192);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int64_t xq = hq * kD + 64 * b, xk = kd + xq, xv = 2 * kd + (int64_t)h * kD + 64 * b;
          if (!STATE && GDN_SPAN_G(xq, 64, a.C)) tma_load_2d(st.qk[b], &xmap, (int32_t)xq, row, &S.full[s]);
          if (GDN_SPAN_G(xk, 64, a.C)) tma_load_2d(st.qk[b] + 8192, &xmap, (int32_t)xk, row, &S.full[s]);
          if (GDN_SPAN_G(xv, 64, a.C)) tma_load_2d(st.v[b], &xmap, (int32_t)xv, row, &S.full[s]);
        }
      }
      __syncwarp();
      ++n_load;
    };
    bool ok = true;
    if (loader) {
      while (n_load < min(nit, kStages - 1)) load();
      // the state tile has passed through the last stage
      if (nit >= kStages && (ok = wait_all(&S.init, 0))) load();
    }
    if (STATE) {
      if (loader)
        for (int i = 0; n_load < nit && ok; ++i)
          if ((ok = wait_all(&S.empty[i % kStages], (i / kStages) & 1))) load();
    } else {
      const int quarter = warp & 3;
      const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);
      const auto out = GDN_GV(reinterpret_cast<__nv_bfloat16*>(a.out), a.total * ld);
      for (int i = 0; i < nit && ok; ++i) {
        const int L = count(i);
        const int64_t at = (S.seg.t0 + from(i)) * ld + (int64_t)h * kD + 32 * quarter + lane;
        if (!(ok = wait_all(&S.o_full, i & 1))) break;
        umma::fence_after();
        if (loader && n_load < nit) load();
        __nv_bfloat162 o[kC / 2];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float o1[8], oh[8], ol[8];
          tmem_ld8x3(tlane + TM_O1 + 8 * c, tlane + TM_O2 + 8 * c, tlane + TM_O2 + kC + 8 * c, o1, oh, ol);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = make_float2(S.ps[8 * c + 2 * e + 1], S.ps[8 * c + 2 * e + 2]);
            o[4 * c + e] = __floats2bfloat162_rn(fmaf(f.x, o1[2 * e], oh[2 * e] + ol[2 * e]),
                                                 fmaf(f.y, o1[2 * e + 1], oh[2 * e + 1] + ol[2 * e + 1]));
          }
        }
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.o_empty);
        // a warp's 32 channels of a token are 64 consecutive bytes
        __nv_bfloat16* const to = &out[at];
        if (L == kC) {
#pragma unroll
          for (int t = 0; t < kC; ++t) to[t * ld] = t & 1 ? o[t / 2].y : o[t / 2].x;
        } else {
#pragma unroll
          for (int t = 0; t < kC; ++t)
            if (t < L) to[t * ld] = t & 1 ? o[t / 2].y : o[t / 2].x;
        }
      }
    }
    if (!ok && lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
    if (loader)  // what is in flight lands before the memory goes (at once, unless a wait expired)
      for (int k = max(0, n_load - kStages); k < n_load; ++k) wait_all(&S.full[k % kStages], (k / kStages) & 1);
  } else {
    // -------------------------------------------------------------------- state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kStateRegs));
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;  // V channel; dk columns 64 half ..
    const uint32_t tlane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int64_t slot_n = ld * kD, own = (int64_t)h * kD * kD;
    const auto pool = GDN_GV(a.ssm, a.num_slots * slot_n);
    const auto segs = GDN_GV(a.seg_state, a.n_segs * slot_n);
    // A tile moves in whole rows (512 bytes per warp access) and through shared
    // memory: piece p of row r at p ^ (r & 7).
    uint8_t* const tile = reinterpret_cast<uint8_t*>(&S.st[kStages - 1]);
    auto piece = [](int r, int p) { return (uint32_t)r * 512u + (uint32_t)((p ^ (r & 7)) << 4); };
    float2 st[32];
    {
      float4 v[16];  // piece `lane` of rows warp, warp + 8, ..
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      auto place = [&](int j) { return own + ((warp + 8 * j) * 32 + lane) * 4; };
      const int seg = S.seg.seg, n_seg = S.seg.n_seg;
      if (seg == 0) {
        const bool kept = !STATE && n_seg > 1;
        const auto src = kept ? GDN_GV((const float*)a.seg_state, a.n_segs * slot_n) + (S.seg.seg0 + n_seg - 1) * slot_n
                              : GDN_GV((const float*)a.ssm, a.num_slots * slot_n) + S.seg.slot * slot_n;
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = vec_at<const float4>(src, place(j));
        if (STATE) {
          const auto keep = segs + (S.seg.seg0 + n_seg - 1) * slot_n;
#pragma unroll
          for (int j = 0; j < 16; ++j) vec_at<float4>(keep, place(j)) = v[j];
        }
      } else if (!STATE) {
        const float dec = power(GDN_GV(a.log_decay, a.hv)[h], (int64_t)a.seg_chunks * kC);
        for (int k = 0; k < seg; ++k) {
          const float d = k ? dec : 0.f;  // the first segment's state holds the slot's already
          const auto from_seg = segs + (S.seg.seg0 + k) * slot_n;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float4 x = vec_at<const float4>(from_seg, place(j));
            v[j].x = fmaf(d, v[j].x, x.x);
            v[j].y = fmaf(d, v[j].y, x.y);
            v[j].z = fmaf(d, v[j].z, x.z);
            v[j].w = fmaf(d, v[j].w, x.w);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) tile_at<float4>(tile, kTile, piece(warp + 8 * j, lane)) = v[j];
      named_sync(1, kStateThreads);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float4 x = tile_at<float4>(tile, kTile, piece(row, 16 * half + e));
        st[2 * e] = lo2(x);
        st[2 * e + 1] = hi2(x);
      }
      umma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.init);
    }
    auto put_s = [&]() {  // the O1 operand
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) split2(st[16 * q + e], hi[e], lo[e]);
        tmem_put16(tlane + TM_SH + 32 * half + 16 * q, hi);
        tmem_put16(tlane + TM_SL + 32 * half + 16 * q, lo);
      }
      tmem_wait_st();
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.s_full);
    };
    if (!STATE) put_s();
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < nit && ok; ++i) {
      const int L = count(i);
      const float dec = S.pw[L];
      if (!(ok = wait_all(&S.ds_full, i & 1))) break;
      umma::fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float d[16];
        umma::tmem_ld16(tlane + TM_DS + 64 * half + 16 * q, d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          st[8 * q + e] = fma2(st[8 * q + e], make_float2(dec, dec), make_float2(d[2 * e], d[2 * e + 1]));
      }
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.ds_empty);
      if (!STATE) {
        if (i + 1 < nit) {
          if (!(ok = wait_all(&S.o_full, i & 1))) break;  // the operand was read
          umma::fence_after();
          put_s();
        }
        // a block boundary at the chunk's end
        const int64_t P = S.seg.p0 + from(i) + L;
        if (a.max_ckpt > 0 && P % a.ckpt_block == 0) {
          const int64_t idx = P / a.ckpt_block - S.seg.p0 / a.ckpt_block - 1;
          if (idx < a.max_ckpt) {
            const int32_t id = GDN_GV(a.ckpt_ids, (long long)a.n_seq * a.max_ckpt)[(int64_t)S.seg.n * a.max_ckpt + idx];
            const int cls = slot_class(id, a.ck_num_slots);
            if (cls == 2 && tid == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
            if (cls == 0) {
              const auto to = GDN_GV(a.ck_ssm, a.ck_num_slots * slot_n) + (id * slot_n + own + row * kD + 64 * half);
              if (((uintptr_t)a.ck_ssm & 31) == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  st_global32(to.at(8 * e, 8), join4(st[4 * e], st[4 * e + 1]), join4(st[4 * e + 2], st[4 * e + 3]));
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) vec_at<float4>(to, 4 * e) = join4(st[2 * e], st[2 * e + 1]);
              }
            }
          }
        }
      }
    }
    if (!STATE && ok) ok = wait_all(&S.drained, 0);  // every product is done: the tile's memory is free
    if (named_sync_or(1, kStateThreads, !ok)) {
      if (tid == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
    } else if (STATE || S.seg.seg == S.seg.n_seg - 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        tile_at<float4>(tile, kTile, piece(row, 16 * half + e)) = join4(st[2 * e], st[2 * e + 1]);
      named_sync(1, kStateThreads);
      const auto to = STATE ? segs + (S.seg.seg0 + S.seg.seg) * slot_n : pool + S.seg.slot * slot_n;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        vec_at<float4>(to, own + ((warp + 8 * j) * 32 + lane) * 4) = tile_at<float4>(tile, kTile, piece(warp + 8 * j, lane));
    }
  }
  umma::fence_before();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(tmem, TM_COLS);
}

}  // namespace

bool chunk_shape(const gdn_dims& d) { return d.dk == kD && d.dv == kD && d.act_dtype == GDN_BF16; }

bool chunk_supported(const gdn_dims& d, int64_t total, const void* qkv, const void* out) {
  return chunk_shape(d) && total > 0 && aligned(qkv, 16) && aligned(out, 16);
}

cudaError_t chunk_launch(const PrefillArgs& a, cudaStream_t s) {
  CUtensorMap xmap;
  cudaError_t e = tensor_map_2d(&xmap, a.qkv, a.total, a.C, 2, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(ChunkSmem) + 1024;
  const dim3 grid(a.hv, a.n_segs);
  if (a.seg_state) {
    constexpr auto k = lin_chunk_kernel<true>;
    if ((e = ssm::allow_smem<k>(smem)) != cudaSuccess) return e;
    if ((e = launch_pdl(k, grid, dim3(kThreads), smem, s, dim3(1), a, xmap)) != cudaSuccess) return e;
  }
  constexpr auto k = lin_chunk_kernel<false>;
  if ((e = ssm::allow_smem<k>(smem)) != cudaSuccess) return e;
  return launch_pdl(k, grid, dim3(kThreads), smem, s, dim3(1), a, xmap);
}

}  // namespace lin
}  // namespace gdn
