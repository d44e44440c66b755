// The state space decode step for large batches (dk = 128, conv width 4):
// persistent CTAs whose copies run ahead of the arithmetic.
//
// HBM bound: a state row of 512 bytes is read and written once, all else is
// about 1 % of it.  One CTA per SM walks items of one request and one QK
// head's group of state rows, whose conv channels it alone reads and writes.
// A producer lane copies the item's conv inputs (history, new row, weights:
// the bundle, two buffers) and its rows (16 KiB pieces through a ring) with
// the copy engine, an item and a ring ahead; eight warps compute features,
// update the rows and store them.  So reads go on through an item's
// prologue, which the split form in ssm.cu leaves to the neighbours on its SM.
// Every wait is bounded; one that expires ends the CTA's work with
// GDN_DEV_ERR_TIMEOUT.
//
// Measured (graph of calls on distinct slots of a large pool, of the copy
// bandwidth): 64 heads of 64 in 8 groups, 56 / 64 / 128 / 256 requests 41.8 /
// 47.9 / 91.9 / 176 us (0.83 / 0.83 / 0.86 / 0.90), the split form 44.7 / 56.3
// / 102 / 183; 32 heads of 128 in 16 groups, 256 requests 180 us (0.88), split
// 188.  Items in halves over clusters of two CTAs, for finer rounds, were
// slower (44.7 / 51.2 / 100 / 194 us): each waits for the other at every item.
#include "ssm.cuh"
#include "decode_tma.cuh"  // sm_count

#include <cstddef>

namespace gdn {
namespace ssm {
namespace {

constexpr int kCW = 8, kCons = kCW * 32, kThr = kCons + 32;  // consumer warps; + the producer
constexpr int kDK = 128, kW = 4;
constexpr int kLPR = kDK / 16;  // lanes per row
constexpr int kRows = 32;       // rows per piece
constexpr int kPiece = kRows * kDK;
constexpr uint32_t kPieceBytes = kPiece * sizeof(float);
constexpr int kMaxRows = 512;   // of a group
constexpr int kMaxListed = 2 * kCons;
constexpr int kMaxCh = 2 * kDK + kMaxRows;
static_assert(kCons == 2 * kDK, "one q or k channel per consumer");

template <typename Tact, typename Tconv, int STAGES>
struct __align__(128) RingSmem {
  float ring[STAGES][kPiece];
  struct __align__(16) Bundle {  // channels q | k | v of the group
    Tconv hist[kW - 1][kMaxCh];
    Tact x[kMaxCh];
    float w[kMaxCh * kW];
    float bias[kMaxCh];
  } bundle[2];
  // by the item's parity, so that one barrier per item is enough
  float qk[2][2 * kDK];
  float row[2][3][kMaxRows];  // dt v, decay, D v
  uint64_t full[STAGES], empty[STAGES], bfull[2], bempty[2];
  int abort;
  int count[2 * kCW];          // usable requests per warp's 32
  uint16_t order[kMaxListed];  // the usable requests
};

template <typename Tact, typename Tconv, int STAGES>
__global__ void __launch_bounds__(kThr, 1) ssm_decode_ring_kernel(const DecodeArgs a) {
  using SM = RingSmem<Tact, Tconv, STAGES>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  SM& S = *reinterpret_cast<SM*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int walks = gridDim.x, rows = a.G * a.dv;
  volatile int* abort_flag = &S.abort;
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], kCW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S.bfull[s], 1);
      mbar_init(&S.bempty[s], kCW);
    }
    S.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const auto ids = GDN_GV(a.slot_ids, a.B);
  // Up to kMaxListed requests: the usable ones are listed, so that padded
  // rows leave no CTA's round empty (61 requests with 5 padded 42 us, 45 if they
  // did).  More: padded rows are passed over in their rounds.
  const bool listed = a.B <= kMaxListed;
  int usable = a.B;
  if (listed) {
    uint32_t m[2] = {0, 0};
    if (warp < kCW) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = e * kCons + tid;
        m[e] = __ballot_sync(0xffffffffu, r < a.B && slot_class(ids[r], a.num_slots) == 0);
        if (lane == 0) S.count[e * kCW + GDN_S(warp, kCW)] = __popc(m[e]);
      }
    }
    __syncthreads();
    usable = 0;
    for (int k = 0; k < 2 * kCW; ++k) {
      if (k % kCW == warp && (m[k / kCW] >> lane & 1))
        S.order[GDN_S(usable + __popc(m[k / kCW] & ((1u << lane) - 1)), kMaxListed)] =
            (uint16_t)(k / kCW * kCons + tid);
      usable += S.count[k];
    }
    __syncthreads();
  }
  const int items = usable * a.hk;
  auto request = [&](int item) { return listed ? (int)S.order[GDN_S(item / a.hk, kMaxListed)] : item / a.hk; };

  if (warp == kCW) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      [[maybe_unused]] const long long ssm_n = (long long)a.num_slots * a.hv * a.dv * kDK,
                                       conv_n = (long long)a.num_slots * (kW - 1) * a.C;
      uint32_t n = 0, vk = 0;
      bool ok = true;
      for (int item = (int)blockIdx.x; item < items && ok && !*abort_flag; item += walks) {
        const int r = request(item), hq = item % a.hk;
        const int32_t slot = ids[r];
        if (slot_class(slot, a.num_slots)) continue;
        const int bb = vk & 1;
        if (!(ok = mbar_wait(&S.bempty[bb], ((vk >> 1) & 1) ^ 1))) break;
        const uint32_t per_ch = 3 * sizeof(Tconv) + sizeof(Tact) + kW * 4 + (a.conv_bias ? 4 : 0);
        mbar_arrive_expect_tx(&S.bfull[bb], per_ch * (2 * kDK + rows));
        auto& B = S.bundle[bb];
        auto g2s = [&](void* dst, const void* src, uint32_t bytes, [[maybe_unused]] const void* base,
                       [[maybe_unused]] long long extent) {
          if (GDN_GBYTES(src, bytes, base, extent) && GDN_SBYTES(dst, bytes, S))
            bulk_g2s(dst, src, bytes, &S.bfull[bb]);
        };
        const Tconv* hist = reinterpret_cast<const Tconv*>(a.conv) + (size_t)slot * (kW - 1) * a.C;
        const Tact* x = reinterpret_cast<const Tact*>(a.qkv) + (size_t)r * a.C;
#pragma unroll
        for (int part = 0; part < 3; ++part) {  // q, k, v
          const size_t c = part < 2 ? (size_t)(part * a.hk + hq) * kDK : 2 * (size_t)a.hk * kDK + (size_t)hq * rows;
          const int at = part * kDK;
          const uint32_t len = part < 2 ? kDK : rows;
          for (int j = 0; j < kW - 1; ++j)
            g2s(&B.hist[j][at], hist + (size_t)j * a.C + c, len * sizeof(Tconv), a.conv, conv_n * sizeof(Tconv));
          g2s(&B.x[at], x + c, len * sizeof(Tact), a.qkv, (long long)a.B * a.C * sizeof(Tact));
          g2s(&B.w[at * kW], a.conv_w + c * kW, len * kW * 4, a.conv_w, (long long)a.C * kW * 4);
          if (a.conv_bias) g2s(&B.bias[at], a.conv_bias + c, len * 4, a.conv_bias, (long long)a.C * 4);
        }
        ++vk;
        const float* src = a.ssm + ((size_t)slot * a.hv + (size_t)hq * a.G) * a.dv * kDK;
        for (int c = 0; c < rows / kRows; ++c, ++n) {
          const int st = n % STAGES;
          if (!(ok = !*abort_flag && mbar_wait(&S.empty[st], ((n / STAGES) & 1) ^ 1))) break;
          mbar_arrive_expect_tx(&S.full[st], kPieceBytes);
          if (GDN_GBYTES(src + (size_t)c * kPiece, kPieceBytes, a.ssm, ssm_n * 4) &&
              GDN_SBYTES(S.ring[GDN_S(st, STAGES)], kPieceBytes, S))
            bulk_g2s(S.ring[st], src + (size_t)c * kPiece, kPieceBytes, &S.full[st]);
        }
      }
      if (!ok || *abort_flag) {  // let what was issued land before the memory goes away
        *abort_flag = 1;
        report(a.err, GDN_DEV_ERR_TIMEOUT);
        for (uint32_t m = n > (uint32_t)STAGES ? n - STAGES : 0; m < n; ++m)
          mbar_wait(&S.full[m % STAGES], (m / STAGES) & 1);
        for (uint32_t m = vk > 2 ? vk - 2 : 0; m < vk; ++m) mbar_wait(&S.bfull[m & 1], (m >> 1) & 1);
      }
    }
  } else {
    // --------------------------------------------------------------- consumers
    const int seg = lane % kLPR, rloc = warp * (32 / kLPR) + lane / kLPR;  // row within a piece
    const auto state = GDN_GV(a.ssm, (long long)a.num_slots * a.hv * a.dv * kDK);
    const auto conv = GDN_GV(reinterpret_cast<Tconv*>(a.conv), (long long)a.num_slots * (kW - 1) * a.C);
    const auto out = GDN_GV(reinterpret_cast<Tact*>(a.out), (long long)a.B * a.hv * a.dv);
    const auto gate_a = GDN_GV(reinterpret_cast<const Tact*>(a.a), (long long)a.B * a.hv);
    uint32_t n = 0, vk = 0;
    bool ok = true;
    // an unusable request's rows are zeros
    auto skip = [&](int r, int hq, int cls) {
      const size_t out0 = ((size_t)r * a.hv + (size_t)hq * a.G) * a.dv;
      if (cls == 2 && hq == 0 && tid == 0) report(a.err, GDN_DEV_ERR_SLOT_OOB);
      for (int i = tid; i < rows; i += kCons) out[out0 + i] = from_f32<Tact>(0.f);
    };
    if (listed && usable < a.B)
      for (int item = blockIdx.x; item < a.B * a.hk; item += walks) {
        const int cls = slot_class(ids[item / a.hk], a.num_slots);
        if (cls) skip(item / a.hk, item % a.hk, cls);
      }
    int32_t slot_next = (int)blockIdx.x < items ? ids[request(blockIdx.x)] : -1;
    for (int item = (int)blockIdx.x; item < items; item += walks) {
      const int r = request(item), hq = item % a.hk;
      const int32_t slot = slot_next;
      if (item + walks < items) slot_next = ids[request(item + walks)];
      const size_t out0 = ((size_t)r * a.hv + (size_t)hq * a.G) * a.dv;
      const int cls = slot_class(slot, a.num_slots);
      if (cls) {
        skip(r, hq, cls);
        continue;
      }
      const int bb = vk & 1;
      // what the gates take, requested before the bundle is waited for
      float ga[2], gl[2], gb[2], gd[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = tid + e * kCons;
        if (i < rows) {
          const int h = hq * a.G + i / a.dv;
          ga[e] = to_f32(gate_a[(size_t)r * a.hv + h]);
          gl[e] = GDN_GV(a.A_log, a.hv)[h];
          gb[e] = GDN_GV(a.dt_bias, a.hv)[h];
          gd[e] = a.D ? GDN_GV(a.D, a.hv)[h] : 0.f;
        }
      }
      // (a warp gives up as one: nothing below may find part of it gone)
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&S.bfull[bb], (vk >> 1) & 1));
      const auto& B = S.bundle[bb];
      Tconv h1, h2, h3;
      auto feature = [&](int i0) -> float {
        const int i = GDN_S(i0, kMaxCh);
        h1 = B.hist[1][i], h2 = B.hist[2][i];
        const float x = to_f32(B.x[i]);
        h3 = from_f32<Tconv>(x);
        const float4 w = *reinterpret_cast<const float4*>(&B.w[i * kW]);
        float acc = a.conv_bias ? B.bias[i] : 0.f;
        acc = fmaf(w.x, to_f32(B.hist[0][i]), acc);
        acc = fmaf(w.y, to_f32(h1), acc);
        acc = fmaf(w.z, to_f32(h2), acc);
        acc = fmaf(w.w, x, acc);
        return silu_f(acc);
      };
      auto shift = [&](size_t c) {  // the history after this token
        const size_t at = (size_t)slot * (kW - 1) * a.C + c;
        conv[at] = h1;
        conv[at + a.C] = h2;
        conv[at + 2 * (size_t)a.C] = h3;
      };
      if (ok) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = tid + e * kCons;
          if (i < rows) {
            const float v = feature(2 * kDK + i);
            shift(2 * (size_t)a.hk * kDK + (size_t)hq * rows + i);
            const Gate g = gate(gl[e], gb[e], ga[e]);
            S.row[bb][0][GDN_S(i, kMaxRows)] = g.dt * v;
            S.row[bb][1][i] = expf(g.g);
            S.row[bb][2][i] = gd[e] * v;
          }
        }
        S.qk[bb][tid] = feature(tid);
        shift((size_t)(tid < kDK ? hq * kDK : (a.hk + hq - 1) * kDK) + tid);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.bempty[bb]);
      if (named_sync_or(1, kCons, !ok)) {
        ok = false;
        break;
      }
      float4 kk[4], qq[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = GDN_S(c * 4 * kLPR + seg * 4, kDK - 3);
        qq[c] = *reinterpret_cast<const float4*>(&S.qk[bb][col]);
        kk[c] = *reinterpret_cast<const float4*>(&S.qk[bb][kDK + col]);
      }
      const auto dst = state + ((size_t)slot * a.hv + (size_t)hq * a.G) * a.dv * kDK;
      for (int c = 0; c < rows / kRows; ++c, ++n) {
        const int st = n % STAGES;
        if (!(ok = __all_sync(0xffffffffu, ok && mbar_wait(&S.full[st], (n / STAGES) & 1)))) break;
        const int row = GDN_S(c * kRows + rloc, kMaxRows);
        const float* src = S.ring[GDN_S(st, STAGES)] + GDN_S(rloc, kRows) * kDK;
        float4 s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = *reinterpret_cast<const float4*>(src + k * 4 * kLPR + seg * 4);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.empty[st]);  // the producer may refill it
        const float dx = S.row[bb][0][row], al = S.row[bb][1][row];
        float o = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[k].x = fmaf(dx, kk[k].x, al * s[k].x);
          s[k].y = fmaf(dx, kk[k].y, al * s[k].y);
          s[k].z = fmaf(dx, kk[k].z, al * s[k].z);
          s[k].w = fmaf(dx, kk[k].w, al * s[k].w);
          st_stream(&vec_at<float4>(dst, (size_t)row * kDK + k * 4 * kLPR + seg * 4), s[k]);
          o += s[k].x * qq[k].x + s[k].y * qq[k].y + s[k].z * qq[k].z + s[k].w * qq[k].w;
        }
#pragma unroll
        for (int m = kLPR / 2; m; m >>= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
        if (seg == 0) out[out0 + row] = from_f32<Tact>(o + S.row[bb][2][row]);
      }
      ++vk;
    }
    if (!ok) {
      *abort_flag = 1;
      report(a.err, GDN_DEV_ERR_TIMEOUT);
    }
  }
}

template <typename Tact, typename Tconv, int STAGES>
cudaError_t launch(const DecodeArgs& a, cudaStream_t s) {
  using SM = RingSmem<Tact, Tconv, STAGES>;
  using B = typename SM::Bundle;
  static_assert(sizeof(SM) <= 227 * 1024, "shared memory of a CTA");
  static_assert(sizeof(B) % 16 == 0 && offsetof(B, x) % 16 == 0 && offsetof(B, w) % 16 == 0 &&
                    offsetof(B, bias) % 16 == 0 && offsetof(SM, bundle) % 16 == 0 && offsetof(SM, qk) % 16 == 0,
                "copies and vectors start 16-byte aligned");
  constexpr auto k = ssm_decode_ring_kernel<Tact, Tconv, STAGES>;
  const cudaError_t e = allow_smem<k>(sizeof(SM));
  if (e != cudaSuccess) return e;
  const int items = a.B * a.hk, sms = sm_count();
  return launch_pdl(k, dim3((unsigned)(items < sms ? items : sms)), dim3(kThr), sizeof(SM), s, dim3(1), a);
}

}  // namespace

bool decode_ring_supported(const gdn_dims& d, int32_t B, const void* qkv, const gdn_ssm_params& p) {
  const int64_t rows = (int64_t)(d.hv / d.hk) * d.dv, C = channels(d);
  if (d.dk != kDK || d.conv_width != kW || rows % kRows || rows > kMaxRows) return false;
  if ((C * (int64_t)dtype_size(d.act_dtype)) % 16 || (C * (int64_t)dtype_size(d.conv_dtype)) % 16) return false;
  return aligned(qkv, 16) && aligned(p.conv_w, 16) && aligned(p.conv_bias, 16) && (int64_t)B * d.hk <= 1 << 30;
}

cudaError_t decode_ring_launch(const DecodeArgs& a, int act, int cv, cudaStream_t s) {
  if (act == GDN_F32) return launch<float, float, 9>(a, s);
  if (cv == GDN_BF16) return launch<__nv_bfloat16, __nv_bfloat16, 10>(a, s);
  return launch<__nv_bfloat16, float, 9>(a, s);
}

}  // namespace ssm
}  // namespace gdn
