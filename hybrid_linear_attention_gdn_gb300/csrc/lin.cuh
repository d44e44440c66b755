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
  // several, a state pass leaves each segment's own state (from zero, the
  // first one from the slot's) in seg_state, the slot's own state at the last
  // segment's otherwise unused place, and each segment starts from its
  // predecessors' states.
  float* seg_state;  // [n_segs][hv][dv][dk]
  int32_t n_segs, seg_chunks;
  // Chunk form: what is in seg_state, and the work's order.  [0]: pieces of work
  // taken; [1 + segment slot hv + head]: whether that place's state is there.
  uint32_t* sync;
  int32_t max_extra;  // most segments beyond the sequences' first ones
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

// sequence n's first segment slot, in 32 bits (a 64-bit division costs as much as
// a load); offsets that are none come out as any number
__device__ __forceinline__ int64_t first_segment(int64_t tokens, int64_t n, int chunks) {
  return (uint32_t)first_slot(tokens, n) / (uint32_t)chunks + n;
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

// One sequence as a lane holds it.
struct Sequence {
  int64_t t0, len, p0;
  int32_t slot;
  bool bad, oob;
};
__device__ __forceinline__ Sequence load_sequence(const PrefillArgs& a, int i) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  Sequence q;
  q.t0 = cu[i];
  q.len = (int64_t)cu[i + 1] - q.t0;
  q.p0 = GDN_GV(a.start_pos, a.n_seq)[i];
  q.slot = GDN_GV(a.slot_ids, a.n_seq)[i];
  q.bad = bad_rows(a, q.t0, q.len, q.p0);
  q.oob = slot_class(q.slot, a.num_slots) == 2;
  return q;
}
__device__ __forceinline__ void report_sequence(const PrefillArgs& a, const Sequence& q) {
  if (q.bad) report(a.err, GDN_DEV_ERR_SEQLENS);
  else if (q.oob) report(a.err, GDN_DEV_ERR_SLOT_OOB);
}
// The first one of a sequence's n_seg segments has what is left of whole ones: it
// waits for no other.  Where the state pass runs beside the others (a.sync), it
// has 7/10 of two segments: the second one waits for a pass over the first, and at
// 1.75 us a block, 0.72 in that pass and some 6 for the hand-over both end at once
// with (1.75 b + 6) / 2.78 of b blocks, 0.69 of 33 and 0.65 of 100.  With it and
// without, 32 heads: seven ragged prompts 56 and 67 us, 2 x 2048 51 and 56, 6000 +
// 2000 90 and 89; 64 heads: 4096 + 100 86 and 99, 8192 161 and 173; 16 heads, 4096 +
// 1000 45 and 44.
__device__ __forceinline__ int64_t first_blocks(const PrefillArgs& a, int64_t blocks, int n_seg, int chunks) {
  const int64_t rest = blocks - (n_seg - 1) * (int64_t)chunks;
  return a.sync && n_seg == 2 ? max(rest, (7 * blocks + 9) / 10) : rest;
}
// segment `seg` of sequence n in segments of `chunks` blocks
__device__ __forceinline__ Segment segment_of(const PrefillArgs& a, const Sequence& q, int n, int64_t seg, int chunks) {
  Segment s;
  const int64_t head = q.p0 % kC;
  s.t0 = q.t0;
  s.p0 = q.p0;
  s.len = q.len;
  s.slot = q.slot;
  s.n = n;
  s.chunks = chunks;
  s.seg0 = first_segment(q.t0, n, chunks);
  s.padded = slot_class(q.slot, a.num_slots) != 0;
  const int64_t blocks = blocks_of(q.len, q.p0);
  s.n_seg = ((uint32_t)blocks + chunks - 1) / (uint32_t)chunks;  // (at most 2^25 + 2 blocks)
  s.seg = (int32_t)seg;
  const int64_t first = first_blocks(a, blocks, s.n_seg, chunks);
  s.m0 = seg ? (first + (seg - 1) * chunks) * kC - head : 0;
  s.m1 = min(q.len, (first + seg * chunks) * kC - head);
  return s;
}

// The segment of segment slot `at`, by one warp or more (every lane gets it).
// false: no such segment.  The leader of segment slot n reports what is wrong
// with sequence n (there are at least as many slots as sequences).
__device__ __forceinline__ bool find_segment(const PrefillArgs& a, const int64_t at, Segment& s, bool leader) {
  const auto cu = GDN_GV(a.cu_seqlens, a.n_seq + 1);
  const int lane = threadIdx.x & 31;
  Sequence q;
  int n;
  if (a.n_seq <= 32) {  // a sequence per lane: one round of loads
    const bool mine = lane < a.n_seq;
    q = load_sequence(a, mine ? lane : 0);
    if (leader && lane == 0 && at < a.n_seq) report_sequence(a, at ? load_sequence(a, (int)at) : q);
    const uint32_t le = __ballot_sync(0xffffffffu, mine && first_segment(q.t0, lane, a.seg_chunks) <= at);
    n = le ? 31 - __clz(le) : 0;
    q.t0 = __shfl_sync(0xffffffffu, q.t0, n);
    q.len = __shfl_sync(0xffffffffu, q.len, n);
    q.p0 = __shfl_sync(0xffffffffu, q.p0, n);
    q.slot = __shfl_sync(0xffffffffu, q.slot, n);
    q.bad = bad_rows(a, q.t0, q.len, q.p0);
  } else {
    if (leader && lane == 0 && at < a.n_seq) report_sequence(a, load_sequence(a, (int)at));
    int lo = 0, m = a.n_seq;  // the answer is in [lo, lo + m)
    while (m > 1) {           // offsets outside [0, total] end this early, never outside the array
      const int step = (m + 31) / 32, i = lane * step;
      const bool le = i < m && first_segment(cu[lo + (i < m ? i : 0)], lo + i, a.seg_chunks) <= at;
      const uint32_t set = __ballot_sync(0xffffffffu, le);
      const int last = set ? 31 - __clz(set) : 0;
      lo += last * step;
      m = min(step, m - last * step);
    }
    n = lo;
    q = load_sequence(a, n);
  }
  if (q.bad) return false;
  const int64_t seg = at - first_segment(q.t0, n, a.seg_chunks);
  s = segment_of(a, q, n, seg, a.seg_chunks);
  return seg >= 0 && seg < s.n_seg;
}

// Piece `item` of the work of at most kMaxCut sequences, by one warp: first the
// state passes of all segments but the last ones, then every sequence's first
// segment, the longest first, then the other segments.  A piece waits for
// earlier ones at most.  Sequences stay whole unless one has cut_from blocks.
// false: there is no such piece.
__device__ __forceinline__ bool find_item(const PrefillArgs& a, int64_t item, Segment& s, bool& state, bool leader) {
  const int lane = threadIdx.x & 31;
  const bool mine = lane < a.n_seq;
  Sequence q = load_sequence(a, mine ? lane : 0);
  if (leader && mine) report_sequence(a, q);
  const int blocks = mine && !q.bad ? (int)blocks_of(q.len, q.p0) : 0;  // (at most 2^25 + 2)
  const int longest = __reduce_max_sync(0xffffffffu, blocks);
  // a sequence without a usable slot has nothing to hand on
  const int chunks = longest < a.cut_from || slot_class(q.slot, a.num_slots) ? (int)kWhole : a.seg_chunks;
  const int n_seg = (blocks + chunks - 1) / chunks, extra = max(n_seg - 1, 0);
  int upto = extra;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const int extras = __shfl_sync(0xffffffffu, upto, 31), firsts = __popc(__ballot_sync(0xffffffffu, n_seg > 0));
  state = item < extras;
  const bool first = !state && item < extras + firsts;
  const int64_t rest = state ? item : item - extras - firsts;  // among those behind the first ones
  uint32_t who;
  if (first) {
    const int key = n_seg ? (int)first_blocks(a, blocks, n_seg, chunks) : 0;
    int rank = 0;
    for (int i = 0; i < a.n_seq; ++i) {
      const int k = __shfl_sync(0xffffffffu, key, i);
      rank += k > key || (k == key && i < lane);
    }
    who = __ballot_sync(0xffffffffu, n_seg > 0 && rank == item - extras);
  } else {
    who = __ballot_sync(0xffffffffu, upto > rest);
  }
  if (!who) return false;
  const int n = __ffs(who) - 1;
  const int before = __shfl_sync(0xffffffffu, upto - extra, n);
  const int64_t seg = first ? 0 : rest - before + (state ? 0 : 1);
  q.t0 = __shfl_sync(0xffffffffu, q.t0, n);
  q.len = __shfl_sync(0xffffffffu, q.len, n);
  q.p0 = __shfl_sync(0xffffffffu, q.p0, n);
  q.slot = __shfl_sync(0xffffffffu, q.slot, n);
  s = segment_of(a, q, n, seg, __shfl_sync(0xffffffffu, chunks, n));
  return true;
}

// lambda^n (n >= 0) as one float, for a factor of a token's own terms: an
// exponent that is rounded (2^-24 of it) hides in what remains of such a term.
// lambda^0 is 1 for every decay, -inf too.
__device__ __forceinline__ float power(float log_decay, int64_t n) {
  return n == 0 ? 1.f : expf(log_decay * (float)n);
}

// A decay as the sum of two floats, for a state that is multiplied by it again
// and again: a rounding to one float (2^-25) is the same every time and adds up,
// over 2,000 remembered multiplications to 6e-5.  As 1 + expm1(log_decay) the
// error is 2^-24 of the small part; a decay that forgets within two
// multiplications needs no second part.
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
// lambda^n, n > 0: of a chunk (2^20 tokens of a memory as long are 16,384 of
// them: with one float the state was 2.1e-4 off) or of a segment
__device__ __forceinline__ Decay decay_of(float log_decay, int64_t n) { return decay_of(log_decay * (float)n); }
// lambda s + x
__device__ __forceinline__ float add_decayed(Decay d, float s, float x) { return fmaf(d.hi, s, fmaf(d.lo, s, x)); }
__device__ __forceinline__ float2 add_decayed2(Decay d, float2 s, float2 x) {
  return fma2(make_float2(d.hi, d.hi), s, fma2(make_float2(d.lo, d.lo), s, x));
}
// lambda s + v k
__device__ __forceinline__ float step(Decay d, float s, float v, float k) { return add_decayed(d, s, v * k); }

__device__ __forceinline__ float2 step2(Decay d, float2 s, float v, float2 k) {
  return add_decayed2(d, s, mul2(make_float2(v, v), k));
}

// words of PrefillArgs::sync
inline int64_t sync_words(int64_t n_segs, int64_t hv) { return 1 + n_segs * hv; }

// The chunk form on the tensor cores (lin_chunk.cu)
bool chunk_shape(const gdn_dims& d);
bool chunk_supported(const gdn_dims& d, int64_t total, const void* qkv, const void* out);
cudaError_t chunk_launch(const PrefillArgs& a, cudaStream_t s);

}  // namespace lin
}  // namespace gdn
