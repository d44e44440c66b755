// Linear attention with a fixed decay per head: pieces shared by its kernels.
#pragma once
#include "gdn_common.cuh"

namespace gdn {
namespace lin {

constexpr int kC = 64;  // tokens per block of absolute positions

struct PrefillArgs {
  float* ssm;
  int32_t num_slots;
  float* ck_ssm;
  int32_t ck_num_slots;
  const float* log_decay;
  float scale;
  const int32_t* slot_ids;
  const int32_t* cu_seqlens;
  const int64_t* start_pos;
  int32_t n_seq;
  int64_t total;
  const int32_t* ckpt_ids;
  int32_t max_ckpt;
  int32_t ckpt_block;
  const void* qkv;
  void* out;
  uint32_t* err;
  int32_t hk, hv, dk, dv, G;
  int64_t C;
  // Segments of seg_chunks blocks; slots n_segs.  Where a sequence has
  // several, a first launch leaves each segment's own state (from zero, the
  // first one from the slot's) in seg_state, the slot's own state at the last
  // segment's otherwise unused place, and a second launch starts each segment
  // from its predecessors' states.
  float* seg_state;  // [n_segs][hv][dv][dk]
  int32_t n_segs, seg_chunks;
};

// Sequence n's blocks occupy the slots from first_slot(cu[n], n) on, its
// segments those from that / seg_chunks + n on.  A sequence of len tokens
// touches at most min(len / 64 + 2, len) blocks, and both of the numbers whose
// smaller one first_slot is grow by at least that much: the ranges are
// disjoint without a scan.
__host__ __device__ __forceinline__ int64_t first_slot(int64_t tokens, int64_t n) {
  const int64_t by_chunk = tokens / kC + 2 * n;
  return by_chunk < tokens ? by_chunk : tokens;
}

// One segment of one sequence.
struct Segment {
  int64_t t0;       // the sequence's first row
  int64_t p0;       // its first position
  int64_t len;      // its tokens
  int64_t seg0;     // its first segment's slot
  int32_t slot, n;  // state slot, sequence
  int32_t seg, n_seg;
  int64_t m0, m1;   // the segment's tokens [m0, m1)
  bool padded;      // no usable slot: outputs are zeros
};

// whether sequence n's rows or positions are inconsistent
__device__ __forceinline__ bool bad_rows(const PrefillArgs& a, int64_t t0, int64_t len, int64_t p0) {
  return t0 < 0 || len < 0 || t0 + len > a.total || p0 < 0 || p0 > INT64_MAX - len - kC;
}

// The segment of segment slot `at`, by one warp or more (every lane gets it).
// false: no such segment.  The leader of segment slot n reports what is wrong
// with sequence n (there are at least as many slots as sequences).
__device__ __forceinline__ bool find_segment(const PrefillArgs& a, const int64_t at, Segment& s, bool leader) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  const int lane = threadIdx.x & 31;
  if (leader && at < a.n_seq) {
    if (bad_rows(a, cu[at], (int64_t)cu[at + 1] - cu[at], GDN_GV(a.start_pos, a.n_seq)[at]))
      report(a.err, GDN_DEV_ERR_SEQLENS);
    else if (slot_class(GDN_GV(a.slot_ids, a.n_seq)[at], a.num_slots) == 2)
      report(a.err, GDN_DEV_ERR_SLOT_OOB);
  }
  int lo = 0, n = a.n_seq;  // the answer is in [lo, lo + n)
  while (n > 1) {           // offsets outside [0, total] end this early, never outside the array
    const int step = (n + 31) / 32, i = lane * step;
    const bool le = i < n && first_slot(cu[lo + (i < n ? i : 0)], lo + i) / a.seg_chunks + (lo + i) <= at;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  s.n = lo;
  s.t0 = cu[lo];
  s.len = (int64_t)cu[lo + 1] - s.t0;
  s.p0 = GDN_GV(a.start_pos, a.n_seq)[lo];
  s.slot = GDN_GV(a.slot_ids, a.n_seq)[lo];
  if (bad_rows(a, s.t0, s.len, s.p0)) return false;
  s.padded = slot_class(s.slot, a.num_slots) != 0;
  s.seg0 = first_slot(s.t0, lo) / a.seg_chunks + lo;
  const int64_t seg = at - s.seg0;
  const int64_t head = s.p0 % kC, nch = s.len ? (head + s.len + kC - 1) / kC : 0;
  s.n_seg = (int32_t)((nch + a.seg_chunks - 1) / a.seg_chunks);
  if (seg < 0 || seg >= s.n_seg) return false;
  s.seg = (int32_t)seg;
  s.m0 = seg ? seg * a.seg_chunks * kC - head : 0;
  s.m1 = min(s.len, (seg + 1) * (int64_t)a.seg_chunks * kC - head);
  return true;
}

// lambda^n (n >= 0).  The rounding of the exponent (2^-24 of it) is the same
// part of every power: what a state still remembers has exponents of a few
// units in sum, however many powers were multiplied.  lambda^0 is 1 for every
// decay, -inf too.
__device__ __forceinline__ float power(float log_decay, int64_t n) {
  return n == 0 ? 1.f : expf(log_decay * (float)n);
}

// A decay as the sum of two floats.  A state that remembers 2,000 tokens has
// been multiplied by lambda as often: its rounding to one float (2^-25) would
// put it off by 6e-5.  As 1 + expm1(log_decay) the error is 2^-24 of the small
// part; a decay that forgets within two tokens needs no second part.
struct Decay {
  float hi, lo;
};
__device__ __forceinline__ Decay decay_of(float log_decay) {
  Decay d;
  const bool slow = log_decay > -0.5f;
  d.hi = slow ? 1.f : expf(log_decay);
  d.lo = slow ? expm1f(log_decay) : 0.f;
  return d;
}
// lambda s + v k
__device__ __forceinline__ float step(Decay d, float s, float v, float k) {
  return fmaf(d.hi, s, fmaf(d.lo, s, v * k));
}

// The chunk form on the tensor cores (lin_chunk.cu)
bool chunk_shape(const gdn_dims& d);
bool chunk_supported(const gdn_dims& d, int64_t total, const void* qkv, const void* out);
cudaError_t chunk_launch(const PrefillArgs& a, cudaStream_t s);

}  // namespace lin
}  // namespace gdn
