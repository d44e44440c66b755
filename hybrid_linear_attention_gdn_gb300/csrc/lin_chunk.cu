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
//   O1^T = S^T Q^T                  A = S^T in TMEM, in parts
//   O2^T = V^T P^T                  A = V; P = G with its decays, in parts
// dS does not need S, so only an elementwise update per chunk is left of the
// recurrence, and the tensor core always has another chunk's work.  lambda^L of
// S's update is two floats (see Decay).
//
// Roundings.  q, k and v are bf16 already and enter G, dS and O2 exactly.  V w
// is split into three bf16 parts (24 bits: the fp32 product itself), so that
// states and checkpoints keep fp32's accuracy; P and S^T, which only outputs
// see, into two (off by at most 2^-17 of a term, against the output's own 2^-8;
// with one part each the outputs were 2.4e-3 off instead of 1.7e-3; a third one,
// for which neither TMEM nor shared memory has room, would be 12 products more a
// chunk).  bf16 parts keep fp32's range (a P or S beyond 3.39e38 is infinite), so
// no scaling is needed.
//
// A product of K = 16 takes some 59 cycles with N = 64 and 67 to 73 with N = 128
// (measured; M = 64 no less than M = 128), 2,630 a chunk, and both operands from
// shared memory take all its bandwidth: two parts of V w therefore go through
// registers to TMEM, whose 512 columns are all in use.
//
// 27 warps by role (of 28): 16 hold S (4 per 32 V channels, 32 dk columns each) and
// make P from G, 4 write outputs, 4 scale and split V (all 8 where there are no
// outputs), one issues the copies and two the products: dS and O1, and G and O2.
// The tensor core takes a product about when the one before it is done, so that one
// issuer's waits for the other warps left it idle a third of the time.
//
// Bound by the products: 2,630 of some 3,100 cycles a chunk, by the products'
// times measured one by one.  In a graph of calls 4 x 8192 tokens of 32 heads 221 us
// (128 CTAs; 0.77 of a copy's rate), 1 x 8192 91 us (five segments), 37 tokens 8.5 us;
// called one by one 235, 91 and 13.  The roles' loops share the instruction
// caches: rolled, and with short waits, their hit rate went from 73 to 94 % and 4 x
// 8192 tokens from 260 to 241 us.
//
// Sequences that may be cut into segments are one launch behind a small one that
// clears the flags: state passes and segments are pieces of work that CTAs take
// in an order in which whatever a piece waits for was taken before it, so that first
// segments and whole sequences run beside the state pass (as two launches: seven
// ragged prompts of 3,968 tokens 71 us, so 63; 2 x 2048 54 and 50; 1 x 8192 93 and 91;
// 2048 alone 36 and 38, the price of the order; all with the decays in one float,
// 1 us less).
#include "lin.cuh"

#include "decode_tma.cuh"  // sm_count
#include "ssm.cuh"         // allow_smem
#include "tma.cuh"
#include "umma.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kD = 128;  // dk = dv
constexpr int kStateWarps = 16, kOutWarp = 16, kSplitWarp = 20, kIssuer = 24, kLoader = 26;  // 24: dS, O1; 25: G, O2
constexpr int kThreads = 28 * 32;
constexpr int kStateThreads = kStateWarps * 32;
// Registers per thread, by warpgroup (four of state, output, split, issuers);
// 896 x 72 at launch is what there is.
constexpr int kLaunchRegs = 72, kStateRegs = 80, kOutRegs = 72, kSplitRegs = 64, kRestRegs = 48;
static_assert(4 * kStateRegs + kOutRegs + kSplitRegs + kRestRegs <= 7 * kLaunchRegs, "the launch's registers");

// TMEM columns.  G (M = 64) is in the first 16 lanes of each warp's 32; S^T and
// V w are two parts each.
constexpr uint32_t TM_G = 0, TM_DS = 64, TM_O1 = 192, TM_O2 = 256, TM_S = 320, TM_VW = 448, TM_COLS = 512;

// Stages of a chunk's inputs, 64-column blocks of 128-byte rows (16-byte piece c
// of row r at c ^ (r & 7)): blocks of q and k rows, then v's; without q smaller
// and more of them: the state pass takes 1,500 cycles a chunk and a copy some
// 2,400, so that three stages had it wait for the copies (1 x 8192 98 -> 93 us,
// with two buffers and two issuers).
template <bool STATE>
struct Stages {
  static constexpr int N = STATE ? 5 : 3;
  static constexpr uint32_t K = STATE ? 0 : 8192, BLOCK = 8192 + K, V = 2 * BLOCK, BYTES = V + 2 * 8192;
  static constexpr int BEFORE_TILE = STATE ? 3 : 2;  // that the state tile leaves free
};
struct __align__(1024) ChunkSmem {
  uint8_t st[Stages<false>::N * Stages<false>::BYTES];
  uint8_t p[2][2][64 * 128];    // P [t][j], by the chunk's parity: its two parts
  uint8_t o[2][64 * 128];       // outputs [t][dv], 64-column blocks
  uint8_t vw[2][64 * 128];      // V w's third part [j][dv], 64-column blocks
  uint8_t ck[kStateWarps][32 * 32];  // a state warp's rows on their way to a checkpoint, 8 columns
  __align__(16) float w[2 * kC];  // lambda^(63 - j), zeros from 64 on
  float ps[kC];                 // scale lambda^n
  float pt[kC];                 // scale lambda^(n + 1)
  Decay dec[kC + 1];            // lambda^n, n > 0
  Segment seg;
  int work, head;
  float log_decay;
  uint64_t full[Stages<true>::N], empty[Stages<true>::N];
  // dsa_go: V w of the chunk's first 32 tokens is there, the last dS has been
  // read; dsb_go: that of its last 32; dsa_done: the former's products are done;
  // o1_go: S is there, the last outputs have been read; o2_go: the latter
  uint64_t dsa_go[2], dsb_go[2], dsa_done[2], ds_full[2];  // by buffer of V w and dS
  uint64_t g_full, p_full, o1_go, o2_go, o_full, init, drained;
  uint32_t tmem_base;
};
// The state tile's way between global memory and the threads' rows: 64 KB from
// kTileAt on, free before the first stage there is loaded and P first written,
// and after the last product (which no output has left by then).
constexpr unsigned kTile = kD * kD * 4, kTileAt = 2 * Stages<false>::BYTES;
static_assert(kTileAt == Stages<true>::BEFORE_TILE * Stages<true>::BYTES, "of whole stages");
static_assert(Stages<true>::N * Stages<true>::BYTES <= offsetof(ChunkSmem, o), "stages without q: P's place, too");
static_assert(sizeof(ChunkSmem) + 1024 <= 232448, "shared memory of a CTA");
static_assert(kTileAt + kTile <= offsetof(ChunkSmem, vw), "state tile");

// The leading 8 bits of both values as bf16, packed in pairs; x: what is left
// of it, exactly.  Three parts hold all of an fp32 value's 24 bits.
__device__ __forceinline__ uint32_t take_bf16(float2& x) {
  const uint32_t u = __float_as_uint(x.x), v = __float_as_uint(x.y);
  x = fma2(make_float2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u)), make_float2(-1.f, -1.f), x);
  return __byte_perm(u, v, 0x7632);
}
__device__ __forceinline__ uint32_t bf16_pair(float2 x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Both values to the nearest bf16, packed in pairs; x: what is left, exactly.
// Two parts (the second one by bf16_pair) are off by at most 2^-17 of the value;
// with a first part by truncation 2^-16, at no less time.
__device__ __forceinline__ uint32_t take_near(float2& x) {
  const uint32_t p = bf16_pair(x);
  x = fma2(make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)), make_float2(-1.f, -1.f), x);
  return p;
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane 8 i + r names row r of
// matrix i; the thread gets (rows 2 (lane % 4), + 1; column lane / 4) of each.
__device__ __forceinline__ void ldmatrix4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void stmatrix4_t(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
// 16 lanes (of `half`: the warp's first or last) x 16 columns: register 2 m + g
// of a thread is lane lane / 4 + 8 g, column 4 m + lane % 4
__device__ __forceinline__ void tmem_put_frag(uint32_t taddr, int half, const uint32_t (&v)[8],
                                              int line = __builtin_LINE()) {
  if (!umma::tmem_ok(taddr, 16, true, line)) return;
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(
          taddr + ((uint32_t)(16 * half) << 16)),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
// the warp's first 16 lanes x 16 columns: register 4 m + 2 g + e of a thread is
// lane lane / 4 + 8 g, column 8 m + 2 (lane % 4) + e
__device__ __forceinline__ void tmem_get_frag(uint32_t taddr, float (&v)[8], int line = __builtin_LINE()) {
  if (!umma::tmem_ok(taddr, 16, true, line)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    return;
  }
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 32 columns of two regions: register 4 m + 2 g + e of a thread is
// lane lane / 4 + 8 g, column 8 m + 2 (lane % 4) + e
__device__ __forceinline__ void tmem_get_frag2(uint32_t ta, uint32_t tb, int half, float (&va)[16], float (&vb)[16],
                                               int line = __builtin_LINE()) {
  if (!umma::tmem_ok(ta, 32, true, line) || !umma::tmem_ok(tb, 32, true, line)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) va[i] = vb[i] = 0.f;
    return;
  }
  const uint32_t off = (uint32_t)(16 * half) << 16;
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%33];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=f"(va[0]), "=f"(va[1]), "=f"(va[2]), "=f"(va[3]), "=f"(va[4]), "=f"(va[5]), "=f"(va[6]), "=f"(va[7]),
      "=f"(va[8]), "=f"(va[9]), "=f"(va[10]), "=f"(va[11]), "=f"(va[12]), "=f"(va[13]), "=f"(va[14]), "=f"(va[15]),
        "=f"(vb[0]), "=f"(vb[1]), "=f"(vb[2]), "=f"(vb[3]), "=f"(vb[4]), "=f"(vb[5]), "=f"(vb[6]), "=f"(vb[7]),
        "=f"(vb[8]), "=f"(vb[9]), "=f"(vb[10]), "=f"(vb[11]), "=f"(vb[12]), "=f"(vb[13]), "=f"(vb[14]), "=f"(vb[15])
      : "r"(ta + off), "r"(tb + off)
      : "memory");
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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Products with a constant accumulate flag, issued in runs by one thread inside
// one branch of a converged warp: 48 cycles each with N = 64, where a predicate
// per product took 59 and a loop over the whole issue code by a single thread
// some 100.
// D (TMEM) (+)= A B, both by descriptor
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                       int line = __builtin_LINE()) {
  if (!umma::tmem_ok(tmem_d, umma::idesc_n(idesc), false, line)) return;
  asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, %4;\n" ::"r"(tmem_d), "l"(a), "l"(b), "r"(idesc),
               "n"((int)ACC)
               : "memory");
}
// the same with A in TMEM (K = 16 values in 8 columns)
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc,
                                       int line = __builtin_LINE()) {
  if (!umma::tmem_ok(tmem_d, umma::idesc_n(idesc), false, line) || !umma::tmem_ok(tmem_a, 8, false, line)) return;
  asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, %4;\n" ::"r"(tmem_d), "r"(tmem_a), "l"(b),
               "r"(idesc), "n"((int)ACC)
               : "memory");
}

// Wait of a whole warp, at most kWaitLimitNs as mbar_wait(), in few
// instructions: the roles' loops share the instruction caches, and a wait's code
// is in all of them.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
  uint32_t t0 = 0;
  while (!__all_sync(0xffffffffu, mbar_test(bar, parity))) {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;\n" : "=r"(t));
    t |= 1;
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, t - t0 > (uint32_t)kWaitLimitNs)) return false;
  }
  return true;
}

// Marks the state at segment slot `at` as there; the writers have met at a barrier.
__device__ __forceinline__ void set_flag(const PrefillArgs& a, int64_t at, int h) {
  __threadfence();
  atomicExch(&GDN_GV(a.sync, 1 + (int64_t)a.n_segs * a.hv)[1 + at * a.hv + h], 1u);
}
// Waits for it, at most kWaitLimitNs; the pieces that set flags wait for none.
__device__ __forceinline__ bool wait_flag(const PrefillArgs& a, int64_t at, int h) {
  const uint32_t* const p = &GDN_GV(a.sync, 1 + (int64_t)a.n_segs * a.hv)[1 + at * a.hv + h];
  uint64_t t0 = 0;
  for (;;) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    if (v) return true;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitLimitNs) return false;
  }
}

// Barriers, before the CTA's own.
template <bool STATE>
__device__ __forceinline__ void init_barriers(ChunkSmem& S) {
  if (threadIdx.x == 64) {
#pragma unroll
    for (int i = 0; i < Stages<STATE>::N; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], STATE ? 1 : 4);  // the products; the warps that see them done
    }
    mbar_init(&S.g_full, 1);
    mbar_init(&S.p_full, kStateWarps + 4);
#pragma unroll
    for (int i = 0; i < (STATE ? 2 : 1); ++i) {
      mbar_init(&S.dsa_go[i], 4 + kStateWarps);
      mbar_init(&S.dsb_go[i], 4);
      mbar_init(&S.dsa_done[i], 1);
      mbar_init(&S.ds_full[i], 1);
    }
    mbar_init(&S.o1_go, kStateWarps + 4);
    mbar_init(&S.o2_go, 4);
    mbar_init(&S.o_full, 2);
    mbar_init(&S.init, kStateWarps);
    mbar_init(&S.drained, 2);
    fence_mbar_init();
  }
}
// A head's factors, before it, too.
__device__ __forceinline__ void init_factors(ChunkSmem& S, const float scale, const float log_decay) {
  const int n = (int)threadIdx.x - 96;
  if (n >= 0 && n < 2 * kC) {
    const float x = n <= kC ? power(log_decay, n) : 0.f;
    if (n >= 1 && n <= kC) S.dec[n] = decay_of(log_decay, n);
    S.w[n < kC ? kC - 1 - n : n] = n < kC ? x : 0.f;
    if (n < kC) S.ps[n] = x * scale;
    if (n >= 1 && n <= kC) S.pt[n - 1] = x * scale;
  }
}

// The chunks of segment S.seg of V head h.  STATE: the segment's own state alone.
template <bool STATE>
__device__ __forceinline__ void run(const PrefillArgs& a, const CUtensorMap& xmap, const CUtensorMap& omap, ChunkSmem& S,
                                    const int h, const int warp) {
  const int tid = threadIdx.x, lane = tid & 31, hq = h / a.G;
  const uint32_t tmem = S.tmem_base;
  // Buffers of V w and dS: one, or two where G, S and the outputs leave their
  // places to the second; chunk i's is buf(i), used for the use(i)-th time.
  auto buf = [](int i) { return STATE ? i & 1 : 0; };
  auto use = [](int i) { return STATE ? i >> 1 : i; };
  auto ds_at = [&](int i) { return tmem + (buf(i) ? TM_O1 : TM_DS); };
  auto vw_at = [&](int i) { return tmem + (buf(i) ? TM_S : TM_VW); };
  using St = Stages<STATE>;
  const int64_t ld = (int64_t)a.hv * kD;
  // chunk i holds the segment's tokens [from(i), from(i) + count(i))
  const int64_t m0 = S.seg.m0, m1 = S.seg.m1;
  const int head = (int)((S.seg.p0 + m0) % kC);  // 0 but for a sequence's first chunk
  const int nit = (int)((m1 - m0 + head + kC - 1) / kC);
  auto from = [&](int i) { return i ? m0 - head + (int64_t)i * kC : m0; };
  auto count = [&](int i) { return (int)(min(m1, m0 - head + (int64_t)(i + 1) * kC) - from(i)); };

  // V w, split: V channels 32 quarter .. + 31 of the chunks' tokens 32 th0 .. 32 th1 - 1,
  // transposed on the way to TMEM, by `threads` threads' warps in all.  A
  // thread's tokens are 8 m + 2 (lane % 4), + 1.
  auto split = [&](const int th0, const int th1, const int threads) {
    const int quarter = warp & 3, j0 = 2 * (lane & 3);
    bool ok = true;
    int i = 0;
    for (; i < nit && ok; ++i) {
      uint8_t* const st = S.st + i % St::N * St::BYTES;
      const int L = count(i);
      ok = wait_all(&S.full[i % St::N], (i / St::N) & 1);
      if (L < kC) {
        if (named_sync_or(2, threads, !ok)) ok = false;
        if (!ok) break;
        // rows behind the chunk are others' values: zeros, or a NaN among them
        // would reach this chunk's products
#pragma unroll 1
        for (int e = tid & (threads - 1); e < (kC - L) * 8; e += threads) {
          const uint32_t at = (uint32_t)(L + e / 8) * 128u + (e % 8) * 16u;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            tile_at<uint4>(st + St::V + 8192 * b, 8192, at) = make_uint4(0, 0, 0, 0);
            tile_at<uint4>(st + St::K + St::BLOCK * b, 8192, at) = make_uint4(0, 0, 0, 0);
          }
        }
        umma::fence_proxy_async();
        named_sync(2, threads);
      }
      if (!ok) break;
      const uint32_t vw_t = vw_at(i) + ((uint32_t)(32 * quarter) << 16);
      const float* const wl = &S.w[kC - L + j0];  // of tokens j0, ..
#pragma unroll 1
      for (int th = th0; th < th1; ++th) {  // 32 tokens
        // the operand was read by the products of the chunk before (STATE: two before)
        if (use(i) > 0 && !(ok = wait_all(th ? &S.ds_full[buf(i)] : &S.dsa_done[buf(i)], (use(i) - 1) & 1))) break;
        umma::fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          // matrices of 8 tokens x 8 channels: lane / 8 = 2 (token group) + channel group
          const int c = 4 * quarter + 2 * half + (lane >> 3 & 1);  // 16-byte piece of the 128 channels
          const int r8 = lane & 7;
          const uint32_t off = (c >> 3) * 8192u + (uint32_t)(32 * th + 8 * (lane >> 4) + r8) * 128u + (((c & 7) ^ r8) << 4);
          const uint32_t row = smem_addr(st + St::V) + off, to = smem_addr(buf(i) ? S.o[0] : S.vw[0]) + off;
          float2 x[8];
#pragma unroll
          for (int m = 0; m < 4; m += 2) {
            uint32_t r[4];
            ldmatrix4_t(row + m * 1024u, r);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[2 * m + k] = make_float2(__uint_as_float(r[k] << 16), __uint_as_float(r[k] & 0xffff0000u));
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float2 w = make_float2(wl[32 * th + 8 * m], wl[32 * th + 8 * m + 1]);
            x[2 * m] = mul2(x[2 * m], w);
            x[2 * m + 1] = mul2(x[2 * m + 1], w);
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t r[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = take_bf16(x[k]);
            tmem_put_frag(vw_t + 32 * part + 16 * th, half, r);
          }
#pragma unroll
          for (int m = 0; m < 4; m += 2) {
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = take_bf16(x[2 * m + k]);
            stmatrix4_t(to + m * 1024u, r);
          }
        }
        umma::fence_proxy_async();
        tmem_wait_st();
        umma::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(th ? &S.dsb_go[buf(i)] : &S.dsa_go[buf(i)]);
      }
      if (!ok) break;
      if (!STATE) {
        // after G(i), so that p_full's phases do not mix: G(i) is issued once
        // P(i - 1) is there
        if (!(ok = wait_all(&S.g_full, i & 1))) break;
        if (lane == 0) mbar_arrive(&S.p_full);
      }
    }
    if (!ok) {
      if (lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
      // a warp whose wait ended just in time may have gone on to a last chunk
      // that is not full: it is not left alone at the barrier there
      if (i < nit - 1 && count(nit - 1) < kC) named_sync_or(2, threads, true);
    }
  };

  if (warp >= kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRestRegs));
    const uint64_t dq0 = umma::desc(smem_addr(S.st), 16, 1024);  // q as rows, k 8 KB on
    bool ok = true;
    int s = 0, s_par = 0;  // a chunk's stage and its phase
    auto next = [&]() {
      if (++s == St::N) {
        s = 0;
        s_par ^= 1;
      }
    };
    if (warp == kIssuer || (STATE && warp == kIssuer + 1)) {
      // -------------- issuer of dS, O1 (STATE: both, of every other chunk's dS)
      constexpr uint32_t ID_DS = umma::idesc_bf16(128, kD, false, true);   // V w in TMEM
      constexpr uint32_t ID_DS3 = umma::idesc_bf16(128, kD, true, true);  // in shared memory
      constexpr uint32_t ID_O1 = umma::idesc_bf16(128, kC, false, false);
      const uint64_t dk0 = umma::desc(smem_addr(S.st) + St::K, St::BLOCK, 1024);  // k as columns
      const uint64_t dvw0 = umma::desc(smem_addr(S.vw[0]), 8192, 1024), dvw1 = umma::desc(smem_addr(S.o[0]), 8192, 1024);
#pragma unroll 1
      for (int i = STATE ? warp - kIssuer : 0; i < nit; i += STATE ? 2 : 1) {
        const uint32_t at = i % St::N * St::BYTES;
        // dS^T = (V w)^T K, the small parts first (whoever split V has seen the
        // chunk's copies land)
        const uint64_t dk = umma::adv(dk0, at), dvw = buf(i) ? dvw1 : dvw0;
        const uint32_t ds = ds_at(i), vw = vw_at(i);
#pragma unroll
        for (int th = 0; th < 2; ++th) {  // 32 tokens, whose V w may be replaced under the others' products
          if (!(ok = wait_all(th ? &S.dsb_go[buf(i)] : &S.dsa_go[buf(i)], use(i) & 1))) break;
          umma::fence_after();
          if (lane == 0) {
#pragma unroll
            for (int k = 2 * th; k < 2 * th + 2; ++k) {
              if (k == 0) mma_ss<false>(ds, dvw, dk, ID_DS3);
              else mma_ss<true>(ds, umma::adv(dvw, 2048 * k), umma::adv(dk, 2048 * k), ID_DS3);
            }
#pragma unroll
            for (int part = 1; part >= 0; --part)
#pragma unroll
              for (int k = 2 * th; k < 2 * th + 2; ++k)
                mma_ts<true>(ds, vw + 32 * part + 8 * k, umma::adv(dk, 2048 * k), ID_DS);
            umma::commit(th ? &S.ds_full[buf(i)] : &S.dsa_done[buf(i)]);
            if (STATE && th) umma::commit(&S.empty[i % St::N]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (!STATE) {
          // O1^T = S^T Q^T
          if (!(ok = wait_all(&S.o1_go, i & 1))) break;
          umma::fence_after();
          if (lane == 0) {
            const uint64_t dq = umma::adv(dq0, at);
            mma_ts<false>(tmem + TM_O1, tmem + TM_S + 64, dq, ID_O1);
#pragma unroll
            for (int k = 1; k < 16; ++k)
              mma_ts<true>(tmem + TM_O1, tmem + TM_S + (k < 8 ? 64 : 0) + 8 * (k & 7),
                           umma::adv(dq, (k >> 2 & 1) * 16384 + (k & 3) * 32), ID_O1);
            umma::commit(&S.o_full);
          }
          __syncwarp();
        }
      }
    } else if (!STATE && warp == kIssuer + 1) {
      // -------------------------------------------------------- issuer of G, O2
      constexpr uint32_t ID_G = umma::idesc_bf16(64, kC, false, false);
      constexpr uint32_t ID_O2 = umma::idesc_bf16(128, kC, true, false);
      const uint64_t dv0 = umma::desc(smem_addr(S.st) + St::V, 8192, 1024);
      const uint64_t dp0 = umma::desc(smem_addr(S.p[0][0]), 16, 1024);
      uint32_t at = 0;  // the stage of the chunk whose G is next
      auto issue_g = [&]() -> bool {
        if (!wait_all(&S.full[s], s_par)) return false;
        umma::fence_after();
        at = s * St::BYTES;
        if (lane == 0) {
          const uint64_t d = umma::adv(dq0, at);
          mma_ss<false>(tmem + TM_G, d, umma::adv(d, 8192), ID_G);
#pragma unroll
          for (int k = 1; k < 8; ++k) {
            const uint32_t o = (k >> 2) * 16384 + (k & 3) * 32;
            mma_ss<true>(tmem + TM_G, umma::adv(d, o), umma::adv(d, 8192 + o), ID_G);
          }
          umma::commit(&S.g_full);
        }
        __syncwarp();
        next();
        return true;
      };
      ok = issue_g();
#pragma unroll 1
      for (int i = 0; i < nit && ok; ++i) {
        const uint64_t dv = umma::adv(dv0, at), dp = umma::adv(dp0, (i & 1) * (uint32_t)sizeof(S.p[0]));
        // P of this chunk is there (G's columns have been read), its V is clean
        if (!(ok = wait_all(&S.p_full, i & 1))) break;
        if (i + 1 < nit && !(ok = issue_g())) break;
        // O2^T = V^T P^T
        if (!(ok = wait_all(&S.o2_go, i & 1))) break;
        umma::fence_after();
        if (lane == 0) {
          mma_ss<false>(tmem + TM_O2, dv, umma::adv(dp, 8192), ID_O2);
#pragma unroll
          for (int k = 1; k < 4; ++k)
            mma_ss<true>(tmem + TM_O2, umma::adv(dv, 2048 * k), umma::adv(dp, 8192 + 32 * k), ID_O2);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ss<true>(tmem + TM_O2, umma::adv(dv, 2048 * k), umma::adv(dp, 32 * k), ID_O2);
          umma::commit(&S.o_full);
        }
        __syncwarp();
      }
    }
    if (warp == kLoader && lane == 0) {
      // ---------------------------------------------------------------- loader
      const int64_t kd = (int64_t)a.hk * kD;
      int n_load = 0;
      for (; n_load < nit; ++n_load) {
        // the state tile has passed through; the products of the stage's last
        // chunk are done (and its V split, which dS waited for)
        if (n_load == St::BEFORE_TILE) ok = mbar_wait(&S.init, 0);
        if (ok && n_load >= St::N) ok = mbar_wait(&S.empty[s], s_par ^ 1);
        if (!ok) break;
        uint8_t* const st = S.st + s * St::BYTES;
        const int32_t row = (int32_t)(S.seg.t0 + from(n_load));
        mbar_arrive_expect_tx(&S.full[s], (STATE ? 4 : 6) * 8192);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int64_t xq = hq * kD + 64 * b, xk = kd + xq, xv = 2 * kd + (int64_t)h * kD + 64 * b;
          if (!STATE && GDN_SPAN_G(xq, 64, a.C)) tma_load_2d(st + St::BLOCK * b, &xmap, (int32_t)xq, row, &S.full[s]);
          if (GDN_SPAN_G(xk, 64, a.C)) tma_load_2d(st + St::K + St::BLOCK * b, &xmap, (int32_t)xk, row, &S.full[s]);
          if (GDN_SPAN_G(xv, 64, a.C)) tma_load_2d(st + St::V + 8192 * b, &xmap, (int32_t)xv, row, &S.full[s]);
        }
        next();
      }
      if (!ok) report(a.err, GDN_DEV_ERR_TIMEOUT);
      // what is in flight lands before the memory goes (at once, unless a wait expired)
      for (int k = max(0, n_load - St::N); k < n_load; ++k) mbar_wait(&S.full[k % St::N], (k / St::N) & 1);
    }
    __syncwarp();
    if (warp <= kIssuer + 1) {
      if (!ok && lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
      // the products in flight end before their memory is used otherwise
      if (lane == 0) umma::commit(&S.drained);
      __syncwarp();
      wait_all(&S.drained, 0);
    }
  } else if (warp >= kSplitWarp) {
    // --------------------------------------------------------------- V w, split
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kSplitRegs));
    split(0, STATE ? 1 : 2, STATE ? 256 : 128);
  } else if (warp >= kOutWarp) {
    // ------------------------------------------------------------------ outputs
    static_assert(kOutRegs == kLaunchRegs, "as at launch");
    if (STATE) {
      split(1, 2, 256);
    } else {
      bool ok = true;
      // V channels 32 quarter .. + 31, transposed on the way to shared memory; a
      // thread's tokens are 8 m + 2 (lane % 4), + 1
      const int quarter = warp & 3;
      const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);
      const bool storer = warp == kOutWarp;
      const auto out = GDN_GV(reinterpret_cast<uint4*>(a.out), a.total * ld / 8);
      if (lane == 0) {  // nothing to read yet
        mbar_arrive(&S.o1_go);
        mbar_arrive(&S.o2_go);
      }
      for (int i = 0; i < nit && ok; ++i) {
        const int L = count(i);
        uint8_t* const ot = S.o[0];
        ok = wait_all(&S.o_full, i & 1);
        umma::fence_after();
        if (lane == 0 && ok) {
          mbar_arrive(&S.empty[i % St::N]);
          if (storer) bulk_wait_read();  // the last chunk's outputs have left their buffer
        }
        if (named_sync_or(3, 128, !ok)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int hc = 0; hc < 4; ++hc) {  // 16 channels x 32 tokens
          // matrices of 8 tokens x 8 channels: lane / 8 = 2 (token group) + channel group
          const int half = hc >> 1, cols = hc & 1, c = 4 * quarter + 2 * half + (lane >> 3 & 1), r8 = lane & 7;
          const uint32_t row = smem_addr(ot) + (c >> 3) * 8192u + (uint32_t)(32 * cols + 8 * (lane >> 4) + r8) * 128u +
                               (((c & 7) ^ r8) << 4);
          float o1[16], o2[16];
          tmem_get_frag2(tlane + TM_O1 + 32 * cols, tlane + TM_O2 + 32 * cols, half, o1, o2);
          if (hc == 3) {
            umma::fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&S.o1_go);
              mbar_arrive(&S.o2_go);
            }
          }
          const float* const f = &S.pt[32 * cols + 2 * (lane & 3)];
#pragma unroll
          for (int m = 0; m < 4; m += 2) {
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 4 * m + 2 * k;
              r[k] = bf16_pair(fma2(*reinterpret_cast<const float2*>(f + 8 * (m + k / 2)), make_float2(o1[e], o1[e + 1]),
                                    make_float2(o2[e], o2[e + 1])));
            }
            stmatrix4_t(row + m * 1024u, r);
          }
        }
        const int64_t t0 = S.seg.t0 + from(i);
        if (L == kC) {
          umma::fence_proxy_async();
          named_sync(3, 128);
          if (storer && lane == 0) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
              if (GDN_SPAN_G((int64_t)h * kD + 64 * b, 64, ld) && GDN_SPAN_G(t0, kC, a.total))
                tma_store_2d(&omap, ot + 8192 * b, (int32_t)((int64_t)h * kD + 64 * b), (int32_t)t0);
          }
        } else {  // rows behind the chunk belong to others
          named_sync(3, 128);
#pragma unroll 1
          for (int e = tid - kOutWarp * 32; e < L * 16; e += 128) {
            const int t = e / 16, c = e % 16;
            out[((t0 + t) * ld + (int64_t)h * kD) / 8 + c] =
                tile_at<uint4>(ot, sizeof(S.o), (c >> 3) * 8192u + t * 128u + (((c & 7) ^ (t & 7)) << 4));
          }
        }
        if (storer && lane == 0) bulk_commit();
        __syncwarp();
      }
      if (storer && lane == 0) bulk_wait_all();
      __syncwarp();
      if (!ok && lane == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
    }
  } else {
    // -------------------------------------------------------------------- state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kStateRegs));
    const int quarter = warp & 3, part = warp >> 2;  // V channels 32 quarter .., dk columns 32 part ..
    const int row = 32 * quarter + lane;
    const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);
    const int64_t slot_n = ld * kD, own = (int64_t)h * kD * kD;
    const auto segs = GDN_GV(a.seg_state, a.n_segs * slot_n);
    // A tile moves in whole rows (512 bytes per warp access) and through shared
    // memory: piece p of row r at p ^ (r & 7).
    uint8_t* const tile = S.st + kTileAt;
    auto piece = [](int r, int p) { return (uint32_t)r * 512u + (uint32_t)((p ^ (r & 7)) << 4); };
    float2 st[16];
    {
      const int seg = S.seg.seg, n_seg = S.seg.n_seg;
      if (!STATE && n_seg > 1) {  // the slot's own state, or the predecessors' passes
        bool there = true;
        if (seg == 0) there = wait_flag(a, S.seg.seg0 + n_seg - 1, h);
        else
          for (int k = lane; k < seg; k += 32) there &= wait_flag(a, S.seg.seg0 + k, h);
        if (!there) report(a.err, GDN_DEV_ERR_TIMEOUT);
        __syncwarp();
      }
      float4 v[8];  // piece `lane` of rows warp, warp + 16, ..
      auto place = [&](int j) { return own + ((warp + 16 * j) * 32 + lane) * 4; };
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (seg == 0) {
        const bool kept = !STATE && n_seg > 1;
        const auto src = kept ? GDN_GV((const float*)a.seg_state, a.n_segs * slot_n) + (S.seg.seg0 + n_seg - 1) * slot_n
                              : GDN_GV((const float*)a.ssm, a.num_slots * slot_n) + S.seg.slot * slot_n;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = vec_at<const float4>(src, place(j));
        if (STATE) {
          const auto keep = segs + (S.seg.seg0 + n_seg - 1) * slot_n;
#pragma unroll
          for (int j = 0; j < 8; ++j) vec_at<float4>(keep, place(j)) = v[j];
        }
      } else if (!STATE) {
        const Decay dec = decay_of(S.log_decay, (int64_t)S.seg.chunks * kC);
        for (int k = 0; k < seg; ++k) {
          const Decay d = k ? dec : Decay{0.f, 0.f};  // the first segment's state holds the slot's already
          const auto from_seg = segs + (S.seg.seg0 + k) * slot_n;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 x = vec_at<const float4>(from_seg, place(j));
            v[j].x = add_decayed(d, v[j].x, x.x);
            v[j].y = add_decayed(d, v[j].y, x.y);
            v[j].z = add_decayed(d, v[j].z, x.z);
            v[j].w = add_decayed(d, v[j].w, x.w);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) tile_at<float4>(tile, kTile, piece(warp + 16 * j, lane)) = v[j];
      named_sync(1, kStateThreads);
      if (STATE && seg == 0 && tid == 0) set_flag(a, S.seg.seg0 + n_seg - 1, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 x = tile_at<float4>(tile, kTile, piece(row, 8 * part + e));
        st[2 * e] = lo2(x);
        st[2 * e + 1] = hi2(x);
      }
      named_sync(1, kStateThreads);
      if (!STATE && part == 0)  // P above the diagonal blocks: zeros, once
        for (int c = 2 * quarter + 2; c < 8; ++c)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            tile_at<uint4>(S.p[b][lane >> 4], sizeof(S.p[0][0]), umma::sw128_off(16 * quarter + (lane & 15), 8 * c, 0)) =
                make_uint4(0, 0, 0, 0);
      umma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.init);
    }
    auto put_s = [&]() {  // the O1 operand
      uint32_t r[16], lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float2 x = st[e];
        r[e] = take_near(x);
        lo[e] = bf16_pair(x);
      }
      tmem_put16(tlane + TM_S + 16 * part, r);
      tmem_put16(tlane + TM_S + 64 + 16 * part, lo);
      tmem_wait_st();
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.o1_go);
    };
    // P: rows 16 quarter .. + 15 (G's first 16 lanes of the quarter), of them
    // the columns 16 part .. + 15, unless they lie above the diagonal; a
    // thread's rows are lane / 4, + 8 and its columns 8 m + 2 (lane % 4), + 1
    auto put_p = [&](int i) {
      if (part <= quarter) {
        float g[8];
        umma::fence_after();
        tmem_get_frag(tlane + TM_G + 16 * part, g);
        const int d0 = 16 * (quarter - part) + (lane >> 2) - 2 * (lane & 3);  // t - j
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // column group k / 2, row group k % 2
          const int d = d0 + 8 * (k & 1) - 8 * (k >> 1), e = 4 * (k >> 1) + 2 * (k & 1);
          float2 x = make_float2(d >= 0 ? g[e] * S.ps[max(d, 0)] : 0.f, d >= 1 ? g[e + 1] * S.ps[max(d - 1, 0)] : 0.f);
          hi[k] = take_near(x);
          lo[k] = bf16_pair(x);
        }
        // matrices of 8 rows x 8 columns: lane / 8 = 2 (column group) + row group.
        // G(i)'s commit covers the products before it, O2(i - 2) among them: P's
        // buffer is free
        const uint32_t to = smem_addr(S.p[i & 1][0]) + (uint32_t)(16 * quarter + (lane & 15)) * 128u +
                            (((2 * part + (lane >> 4)) ^ (lane & 7)) << 4);
        stmatrix4(to, hi);
        stmatrix4(to + 8192u, lo);
        umma::fence_proxy_async();
        umma::fence_before();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(&S.p_full);
    };
    if (!STATE) put_s();
    if (lane == 0) {  // no dS to read yet
      mbar_arrive(&S.dsa_go[0]);
      if (STATE) mbar_arrive(&S.dsa_go[1]);
    }
    bool ok = true;
    if (!STATE && (ok = wait_all(&S.g_full, 0))) put_p(0);
    // the chunk that ends at the next block boundary, and the boundary's place
    const int kpc = a.ckpt_block / kC;
    int to_ckpt = nit;
    int64_t ck_idx = 0;
    if (!STATE && a.max_ckpt > 0) {
      const int64_t c0 = (S.seg.p0 + m0) / kC;  // the first chunk's absolute number
      to_ckpt = kpc - 1 - (int)(c0 % kpc);
      ck_idx = c0 / kpc - S.seg.p0 / a.ckpt_block;
    }
#pragma unroll 1
    for (int i = 0; i < nit && ok; ++i) {
      const int L = count(i);
      const Decay dec = S.dec[L];
      // the decay is applied under the wait for dS: 4 x 8192 tokens 224 us in a
      // graph, with both of its factors behind the wait 227 (with one rounded factor 222)
      if (dec.hi == 1.f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) st[e] = fma2(make_float2(dec.lo, dec.lo), st[e], st[e]);
      } else {  // (no second part)
#pragma unroll
        for (int e = 0; e < 16; ++e) st[e] = mul2(make_float2(dec.hi, dec.hi), st[e]);
      }
      if (!(ok = wait_all(&S.ds_full[buf(i)], use(i) & 1))) break;
      umma::fence_after();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float d[16];
        umma::tmem_ld16(ds_at(i) + ((uint32_t)(32 * quarter) << 16) + 32 * part + 16 * q, d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          st[8 * q + e] = fma2(st[8 * q + e], make_float2(1.f, 1.f), make_float2(d[2 * e], d[2 * e + 1]));
      }
      umma::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.dsa_go[buf(i)]);
      if (!STATE) {
        if (i + 1 < nit) {
          if (!(ok = wait_all(&S.g_full, (i + 1) & 1))) break;
          put_p(i + 1);
          if (!(ok = wait_all(&S.o_full, i & 1))) break;  // the operand was read
          umma::fence_after();
          put_s();
        }
        // a block boundary at the chunk's end (a sequence that ends inside the
        // chunk does not reach it)
        if (i == to_ckpt) {
          to_ckpt += kpc;
          const bool whole = i + 1 < nit || (S.seg.p0 + m1) % kC == 0;
          if (whole && ck_idx < a.max_ckpt) {
            const int32_t id =
                GDN_GV(a.ckpt_ids, (long long)a.n_seq * a.max_ckpt)[(int64_t)S.seg.n * a.max_ckpt + ck_idx];
            const int cls = slot_class(id, a.ck_num_slots);
            if (cls == 2 && tid == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
            if (cls == 0) {
              // 8 columns at a time through the warp's 1 KB: 32-byte runs of 16
              // rows per access
              const auto to = GDN_GV(a.ck_ssm, a.ck_num_slots * slot_n) + (id * slot_n + own + (row - lane) * kD + 32 * part);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  tile_at<float4>(S.ck[warp], sizeof(S.ck[0]), (uint32_t)lane * 32u + ((e ^ (lane >> 2 & 1)) << 4)) =
                      join4(st[4 * q + 2 * e], st[4 * q + 2 * e + 1]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int r = 16 * j + lane / 2;
                  vec_at<float4>(to, r * kD + 8 * q + 4 * (lane & 1)) =
                      tile_at<float4>(S.ck[warp], sizeof(S.ck[0]), (uint32_t)r * 32u + (((lane & 1) ^ (r >> 2 & 1)) << 4));
                }
                __syncwarp();
              }
            }
          }
          ++ck_idx;
        }
      }
    }
    if (!STATE && ok) ok = wait_all(&S.drained, 0);  // every product is done: the tile's memory is free
    if (named_sync_or(1, kStateThreads, !ok)) {
      if (tid == 0) report(a.err, GDN_DEV_ERR_TIMEOUT);
    } else if (STATE || S.seg.seg == S.seg.n_seg - 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        tile_at<float4>(tile, kTile, piece(row, 8 * part + e)) = join4(st[2 * e], st[2 * e + 1]);
      named_sync(1, kStateThreads);
      const auto to = STATE ? segs + (S.seg.seg0 + S.seg.seg) * slot_n
                            : GDN_GV(a.ssm, a.num_slots * slot_n) + S.seg.slot * slot_n;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        vec_at<float4>(to, own + ((warp + 16 * j) * 32 + lane) * 4) = tile_at<float4>(tile, kTile, piece(warp + 16 * j, lane));
    }
    if (STATE) {
      named_sync(1, kStateThreads);
      if (tid == 0) set_flag(a, S.seg.seg0 + S.seg.seg, h);  // (after a timeout, too: nobody waits for long)
    }
  }
}

// CUT: some sequences may be cut into segments.  A CTA takes the next piece of
// work, state passes before the segments that wait for them, so that whatever is
// waited for has begun.  Else grid (V heads, sequences).
template <bool CUT>
__global__ void __launch_bounds__(kThreads, 1)
    lin_chunk_kernel(const PrefillArgs a, const __grid_constant__ CUtensorMap xmap,
                     const __grid_constant__ CUtensorMap omap) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  ChunkSmem& S = *reinterpret_cast<ChunkSmem*>(smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one value per warp
  if (warp == 1) umma::tmem_alloc(&S.tmem_base, TM_COLS);
  if (!CUT) init_barriers<false>(S);
  pdl_wait();
  pdl_trigger();
  if (!CUT && tid >= 96 && tid < 96 + 2 * kC) init_factors(S, a.scale, GDN_GV(a.log_decay, a.hv)[blockIdx.x]);
  if (warp == 0) {
    Segment s;
    bool some, state = false;
    int h = blockIdx.x;
    float log_decay;
    if (CUT) {
      uint32_t ticket = 0;
      if (lane == 0) ticket = atomicAdd(&GDN_GV(a.sync, 1)[0], 1u);
      ticket = __shfl_sync(0xffffffffu, ticket, 0);
      h = (int)(ticket % a.hv);
      log_decay = GDN_GV(a.log_decay, a.hv)[h];
      some = find_item(a, ticket / a.hv, s, state, ticket == 0);
    } else {
      log_decay = GDN_GV(a.log_decay, a.hv)[h];
      some = find_segment(a, blockIdx.y, s, lane == 0 && h == 0);
    }
    if (lane == 0) {
      S.seg = s;
      S.head = h;
      S.work = !some ? 0 : state ? 1 : s.padded ? 2 : 3;
      S.log_decay = log_decay;
    }
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const int work = S.work, h = CUT ? S.head : (int)blockIdx.x;
  if (work == 3) {
    if (CUT) {
      init_barriers<false>(S);
      init_factors(S, a.scale, S.log_decay);
      __syncthreads();
    }
    run<false>(a, xmap, omap, S, h, warp);
  } else if (CUT && work == 1) {
    init_barriers<true>(S);
    init_factors(S, a.scale, S.log_decay);
    __syncthreads();
    run<true>(a, xmap, omap, S, h, warp);
  } else if (work == 2) {  // outputs of an unusable slot: zeros
    const int64_t ld = (int64_t)a.hv * kD;
    const auto out = GDN_GV(reinterpret_cast<uint4*>(a.out), a.total * ld / 8);
    const int64_t n = (S.seg.m1 - S.seg.m0) * (kD / 8);
    for (int64_t e = tid; e < n; e += kThreads)
      out[((S.seg.t0 + S.seg.m0 + e / (kD / 8)) * ld + (int64_t)h * kD) / 8 + e % (kD / 8)] = make_uint4(0, 0, 0, 0);
  }
  umma::fence_before();
  __syncthreads();
  if (warp == 1) umma::tmem_dealloc(S.tmem_base, TM_COLS);
}

// no piece taken, no state there
__global__ void __launch_bounds__(256) lin_clear_kernel(uint32_t* sync, int64_t words) {
  pdl_wait();
  pdl_trigger();
  const auto w = GDN_GV(sync, words);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) w[i] = 0;
}

}  // namespace

bool chunk_shape(const gdn_dims& d) { return d.dk == kD && d.dv == kD && d.act_dtype == GDN_BF16; }

bool chunk_supported(const gdn_dims& d, int64_t total, const void* qkv, const void* out) {
  return chunk_shape(d) && total > 0 && aligned(qkv, 16) && aligned(out, 16);
}

cudaError_t chunk_launch(const PrefillArgs& a, cudaStream_t s) {
  CUtensorMap xmap, omap;
  cudaError_t e = tensor_map_2d(&xmap, a.qkv, a.total, a.C, 2, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  if ((e = tensor_map_2d(&omap, a.out, a.total, (int64_t)a.hv * kD, 2, 64, kC, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
    return e;
  const size_t smem = sizeof(ChunkSmem) + 1024;
  if (a.seg_state) {
    const int64_t words = sync_words(a.n_segs, a.hv);
    const int64_t pieces = (2LL * a.max_extra + a.n_seq) * a.hv;  // state passes, segments behind the first ones, those
    if ((e = launch_pdl(lin_clear_kernel, dim3((unsigned)std::min<int64_t>((words + 255) / 256, 64)), dim3(256), 0, s,
                        dim3(1), a.sync, words)) != cudaSuccess)
      return e;
    constexpr auto k = lin_chunk_kernel<true>;
    if ((e = ssm::allow_smem<k>(smem)) != cudaSuccess) return e;
    return launch_pdl(k, dim3((unsigned)pieces), dim3(kThreads), smem, s, dim3(1), a, xmap, omap);
  }
  constexpr auto k = lin_chunk_kernel<false>;
  if ((e = ssm::allow_smem<k>(smem)) != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.hv, a.n_segs), dim3(kThreads), smem, s, dim3(1), a, xmap, omap);
}

}  // namespace lin
}  // namespace gdn
