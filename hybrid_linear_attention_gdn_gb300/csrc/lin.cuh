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
  // > 0 (at most kMaxCut sequences): they stay whole unless one has this many
  // blocks, which only the device knows
  int32_t cut_from;
};

constexpr int64_t kWhole = 1 << 30;  // blocks of a segment where sequences stay whole
constexpr int kMaxCut = 32;

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
  int32_t chunks;   // blocks per segment
  int64_t m0, m1;   // the segment's tokens [m0, m1)
  bool padded;      // no usable slot: outputs are zeros
};

// whether sequence n's rows or positions are inconsistent
__device__ __forceinline__ bool bad_rows(const PrefillArgs& a, int64_t t0, int64_t len, int64_t p0) {
  return t0 < 0 || len < 0 || t0 + len > a.total || p0 < 0 || p0 > INT64_MAX - len - kC;
}

// blocks of absolute positions that len tokens from position p0 on touch
__device__ __forceinline__ int64_t blocks_of(int64_t len, int64_t p0) { return len ? (p0 % kC + len + kC - 1) / kC : 0; }

// The segment of segment slot `at`, by one warp or more (every lane gets it).
// false: no such segment.  The leader of segment slot n reports what is wrong
// with sequence n (there are at least as many slots as sequences).
__device__ __forceinline__ bool find_segment(const PrefillArgs& a, const int64_t at, Segment& s, bool leader) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1), ids = GDN_GV(a.slot_ids, a.n_seq);
  const auto start = GDN_GV(a.start_pos, a.n_seq);
  const int lane = threadIdx.x & 31;
  s.chunks = a.seg_chunks;
  bool bad;
  if (a.n_seq <= 32) {  // a sequence per lane: one round of loads
    const bool mine = lane < a.n_seq;
    const int i = mine ? lane : 0;
    const int64_t t0 = cu[i], len = (int64_t)cu[i + 1] - t0, p0 = start[i];
    const int32_t slot = ids[i];
    bad = bad_rows(a, t0, len, p0);
    const bool oob = slot_class(slot, a.num_slots) == 2;
    if (a.cut_from > 0) {
      // (a sequence has at most 2^25 + 2 blocks)
      const int longest = __reduce_max_sync(0xffffffffu, mine && !bad ? (int)blocks_of(len, p0) : 0);
      if (longest < a.cut_from) s.chunks = (int32_t)kWhole;
    }
    const uint32_t bad_set = __ballot_sync(0xffffffffu, mine && bad), oob_set = __ballot_sync(0xffffffffu, mine && oob);
    if (leader && at < a.n_seq) {
      if (bad_set >> at & 1) report(a.err, GDN_DEV_ERR_SEQLENS);
      else if (oob_set >> at & 1) report(a.err, GDN_DEV_ERR_SLOT_OOB);
    }
    s.seg0 = first_slot(t0, i) / s.chunks + i;
    const uint32_t le = __ballot_sync(0xffffffffu, mine && s.seg0 <= at);
    s.n = le ? 31 - __clz(le) : 0;
    bad = bad_set >> s.n & 1;
    s.t0 = __shfl_sync(0xffffffffu, t0, s.n);
    s.len = __shfl_sync(0xffffffffu, len, s.n);
    s.p0 = __shfl_sync(0xffffffffu, p0, s.n);
    s.slot = __shfl_sync(0xffffffffu, slot, s.n);
    s.seg0 = __shfl_sync(0xffffffffu, s.seg0, s.n);
  } else {
    if (leader && at < a.n_seq) {
      if (bad_rows(a, cu[at], (int64_t)cu[at + 1] - cu[at], start[at])) report(a.err, GDN_DEV_ERR_SEQLENS);
      else if (slot_class(ids[at], a.num_slots) == 2) report(a.err, GDN_DEV_ERR_SLOT_OOB);
    }
    int lo = 0, n = a.n_seq;  // the answer is in [lo, lo + n)
    while (n > 1) {           // offsets outside [0, total] end this early, never outside the array
      const int step = (n + 31) / 32, i = lane * step;
      const bool le = i < n && first_slot(cu[lo + (i < n ? i : 0)], lo + i) / s.chunks + (lo + i) <= at;
      const uint32_t m = __ballot_sync(0xffffffffu, le);
      const int last = m ? 31 - __clz(m) : 0;
      lo += last * step;
      n = min(step, n - last * step);
    }
    s.n = lo;
    s.t0 = cu[lo];
    s.len = (int64_t)cu[lo + 1] - s.t0;
    s.p0 = start[lo];
    s.slot = ids[lo];
    bad = bad_rows(a, s.t0, s.len, s.p0);
    s.seg0 = first_slot(s.t0, lo) / s.chunks + lo;
  }
  if (bad) return false;
  s.padded = slot_class(s.slot, a.num_slots) != 0;
  const int64_t seg = at - s.seg0, head = s.p0 % kC;
  s.n_seg = (int32_t)((blocks_of(s.len, s.p0) + s.chunks - 1) / s.chunks);
  if (seg < 0 || seg >= s.n_seg) return false;
  s.seg = (int32_t)seg;
  s.m0 = seg ? seg * s.chunks * kC - head : 0;
  s.m1 = min(s.len, (seg + 1) * (int64_t)s.chunks * kC - head);
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

__device__ __forceinline__ float2 step2(Decay d, float2 s, float v, float2 k) {
  return fma2(make_float2(d.hi, d.hi), s, fma2(make_float2(d.lo, d.lo), s, mul2(make_float2(v, v), k)));
}

// The chunk form on the tensor cores (lin_chunk.cu)
bool chunk_shape(const gdn_dims& d);
bool chunk_supported(const gdn_dims& d, int64_t total, const void* qkv, const void* out);
cudaError_t chunk_launch(const PrefillArgs& a, cudaStream_t s);

}  // namespace lin
}  // namespace gdn
