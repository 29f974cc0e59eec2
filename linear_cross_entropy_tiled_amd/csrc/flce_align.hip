// Preference and policy losses over per-token log-probabilities.
//
// Both are one pass over the tokens (a few fp32 operations per 4 to 20 bytes:
// bound by memory, or by launch latency below about a million tokens), a merge
// of per-wave partial sums, and in the backward one pass that writes the
// gradient.  Work is cut by tokens, not by sequences: a wave takes one chunk of
// C consecutive tokens, so one long sequence spreads over the chip and many
// short ones share a wave.
//
// Per-sequence sums without atomics: walking the tokens in order, each step
// moves on by one chunk or one sequence, so the pairs (chunk c, sequence s) that
// meet form a staircase, and c + s names each pair uniquely.  The wave of chunk
// c leaves its partial sum of sequence s in slot c + s; a sequence's sum is its
// slots c0 + s .. c1 + s, added in chunk order.  Padded rows have whole chunks of
// their own: slot = row * chunks_per_row + c.
//
// Sums are fp64 from the first addition: a sequence's log-probability is a sum
// of thousands of terms of one sign, and the preference loss uses the difference
// of two of them.
#include "flce_align.h"
#include "flce_device.h"

namespace flce {

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

__device__ __forceinline__ int64_t load_offset(const Seqs& q, int64_t i) {
  const int64_t v = q.off_i32 ? (int64_t) reinterpret_cast<const int32_t*>(q.offsets)[i]
                              : reinterpret_cast<const int64_t*>(q.offsets)[i];
  return v < 0 ? 0 : (v > q.length ? q.length : v);   // whatever they hold, no access leaves the buffers
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int64_t readlane64(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)v >> 32), lane);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The sequence a wave's walk along the packed tokens is in: the last s with
// offsets[s] <= t (-1 before the first, S behind the last).  64 offsets at a time
// are held one per lane.
struct SeqWalk {
  int64_t s, base, win;

  __device__ __forceinline__ void fill(const Seqs& q, int64_t at, int lane) {
    base = at;
    win = load_offset(q, at + lane < q.S ? at + lane : q.S);
  }
  __device__ __forceinline__ int64_t offset(const Seqs& q, int64_t i, int lane) {
    if (i < base || i >= base + 64) fill(q, i, lane);
    return readlane64(win, (int)(i - base));
  }
  // first token of the next sequence
  __device__ __forceinline__ int64_t next(const Seqs& q, int lane) {
    return s < q.S ? offset(q, s + 1, lane) : INT64_MAX;
  }
  // 64-way search: three rounds reach 262144 sequences
  __device__ __forceinline__ void seek(const Seqs& q, int64_t t, int lane) {
    int64_t first = 0, n = q.S + 1;
    while (n > 64) {
      const int64_t step = (n + 63) / 64, i = (lane + 1) * step - 1;
      const bool below = i < n && load_offset(q, first + i) <= t;
      const int c = __popcll(__builtin_amdgcn_ballot_w64(below));
      first += c * step;
      n = n - c * step < step ? n - c * step : step;
    }
    const bool below = lane < n && load_offset(q, first + lane) <= t;
    s = uniform64(first) + __popcll(__builtin_amdgcn_ballot_w64(below)) - 1;
    fill(q, s < 0 ? 0 : s, lane);
  }
};

// Where a wave's chunk lies.
struct Chunk {
  int64_t row, begin, end;   // tokens [begin, end) of row (packed: row 0)
};
__device__ __forceinline__ Chunk wave_chunk(const Seqs& q, int64_t w) {
  Chunk c;
  c.row = q.packed ? 0 : w / q.chunks_per_row;
  c.begin = (q.packed ? w : w - c.row * q.chunks_per_row) * q.chunk;
  c.end = c.begin + q.chunk < q.length ? c.begin + q.chunk : q.length;
  return c;
}

// The 256 tokens of one step, four to a lane: consecutive ones where they are
// loaded as vectors, else 64 apart, so that every load instruction reads one run.
template <bool VEC> __device__ __forceinline__ int tok(int j, int lane) { return VEC ? 4 * lane + j : 64 * j + lane; }

template <typename T> struct Vec4;
template <> struct Vec4<float> { typedef f32x4 type; };
template <> struct Vec4<bf16> { typedef bf16x4 type; };
template <> struct Vec4<f16> { typedef f16x4 type; };

// p points at the step's first token; tokens at n or later are not read (0).
template <typename T, bool VEC>
__device__ __forceinline__ void load_tokens(const T* p, int n, int lane, float* out) {
  if (VEC && tok<true>(3, lane) < n) {
    const typename Vec4<T>::type v = *reinterpret_cast<const typename Vec4<T>::type*>(p + 4 * lane);
#pragma unroll
    for (int j = 0; j < 4; j++) out[j] = (float)v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) out[j] = tok<VEC>(j, lane) < n ? (float)p[tok<VEC>(j, lane)] : 0.0f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_tokens(T* p, int n, int lane, const float* v) {
  if (VEC && tok<true>(3, lane) < n) {
    typename Vec4<T>::type o;
#pragma unroll
    for (int j = 0; j < 4; j++) o[j] = (T)v[j];
    *reinterpret_cast<typename Vec4<T>::type*>(p + 4 * lane) = o;
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (tok<VEC>(j, lane) < n) p[tok<VEC>(j, lane)] = (T)v[j];
  }
}
// The lane's four mask bytes, one above the other.
template <bool VEC> __device__ __forceinline__ uint32_t load_mask(const uint8_t* p, int n, int lane) {
  if (VEC && tok<true>(3, lane) < n) return *reinterpret_cast<const uint32_t*>(p + 4 * lane);
  uint32_t v = 0;
#pragma unroll
  for (int j = 0; j < 4; j++)
    if (tok<VEC>(j, lane) < n) v |= (uint32_t)p[tok<VEC>(j, lane)] << (8 * j);
  return v;
}

// A step's inputs: up to K token tensors and the mask, loaded one step ahead of their
// use (a step's arithmetic is short next to a load's latency).
template <int K> struct StepIn {
  float x[K][4];
  uint32_t mask;
};

// The step's tokens: which count, and (packed, when `walk` is used) in which
// sequence each lies.  Moves the walk to the sequence of the step's last token.
template <bool PACKED, bool VEC>
__device__ __forceinline__ void step_tokens(const Seqs& q, const Chunk& c, int64_t t, int n, uint32_t mask, bool by_seq,
                                            SeqWalk& walk, int64_t first, int64_t last, int lane, bool (&keep)[4],
                                            int64_t (&seq)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int64_t at = t + tok<VEC>(j, lane);
    keep[j] = tok<VEC>(j, lane) < n && (!PACKED || (at >= first && at < last)) && ((mask >> (8 * j)) & 0xFF) != 0;
    seq[j] = PACKED ? walk.s : c.row;
  }
  if (PACKED && by_seq) {
    for (int64_t edge = walk.next(q, lane); edge < t + n; edge = walk.next(q, lane)) {
      walk.s++;
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (t + tok<VEC>(j, lane) >= edge) seq[j] = walk.s;
    }
    // (offsets that decrease, against the rules, may lead the search past the last sequence)
#pragma unroll
    for (int j = 0; j < 4; j++) keep[j] = keep[j] && seq[j] >= 0 && seq[j] < q.S;
  }
}

// Tokens of the step at t (0 past the chunk), and their mask bytes (no mask: all set).
__device__ __forceinline__ int step_size(const Chunk& c, int64_t t) {
  return (int)(c.end - t < 256 ? (c.end > t ? c.end - t : 0) : 256);
}
template <bool VEC> __device__ __forceinline__ uint32_t step_mask(const Seqs& q, const Chunk& c, int64_t t, int n, int lane) {
  return q.mask ? load_mask<VEC>(q.mask + c.row * q.ld_mask + t, n, lane) : 0x01010101u;
}

// Running sum of the sequence a wave is in, and its flush into a slot.
struct SeqSum {
  double sum;
  int count;

  __device__ __forceinline__ void clear() {
    sum = 0.0;
    count = 0;
  }
  __device__ __forceinline__ void flush(SeqPart* slot, int lane) {
    const double s = wave_sum(sum);
    const int n = wave_sum(count);
    if (lane == 0) {
      slot->sum = s;
      slot->count = n;
    }
    clear();
  }
  // adds the step's values; sequences from .. to lie in the step, and every one
  // but the last ends in it
  __device__ __forceinline__ void add(const Seqs& q, SeqPart* slots, int64_t w, int64_t from, int64_t to,
                                      const bool (&keep)[4], const int64_t (&seq)[4], const float (&v)[4], int lane) {
    for (int64_t s = from;; s++) {
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (keep[j] && (from == to || seq[j] == s)) {
          sum += (double)v[j];
          count++;
        }
      if (s >= to) break;
      if (s >= 0) flush(slots + w + s, lane);
      else clear();
    }
  }
};

// ---------------------------------------------------------------------------
// Preference loss
// ---------------------------------------------------------------------------
template <typename T, bool PACKED, bool VEC>
__global__ __launch_bounds__(256) void preference_tokens_kernel(PreferenceArgs a) {
  const Seqs& q = a.q;
  const int lane = lane_id();
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= q.waves) return;
  const Chunk c = wave_chunk(q, w);
  const int64_t first = PACKED ? load_offset(q, 0) : 0, last = PACKED ? load_offset(q, q.S) : 0;
  SeqWalk walk;
  walk.s = 0;
  if (PACKED) walk.seek(q, c.begin, lane);
  SeqSum acc;
  acc.clear();
  const T* lp = reinterpret_cast<const T*>(a.logps) + c.row * a.ld_logps;
  const T* ref = a.ref ? reinterpret_cast<const T*>(a.ref) + c.row * a.ld_ref : nullptr;
  auto load = [&](int64_t t, StepIn<2>& in) {
    const int n = step_size(c, t);
    load_tokens<T, VEC>(lp + t, n, lane, in.x[0]);
    if (ref) load_tokens<T, VEC>(ref + t, n, lane, in.x[1]);
    in.mask = step_mask<VEC>(q, c, t, n, lane);
  };
  StepIn<2> in, ahead;
  load(c.begin, in);
  for (int64_t t = c.begin; t < c.end; t += 256, in = ahead) {
    load(t + 256, ahead);
    const int n = step_size(c, t);
    bool keep[4];
    int64_t seq[4];
    const int64_t from = walk.s;
    step_tokens<PACKED, VEC>(q, c, t, n, in.mask, true, walk, first, last, lane, keep, seq);
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = ref ? in.x[0][j] - in.x[1][j] : in.x[0][j];
    acc.add(q, a.slots, w, from, PACKED ? walk.s : from, keep, seq, x, lane);
  }
  if (PACKED) {
    if (walk.s >= 0 && walk.s < q.S) acc.flush(a.slots + w + walk.s, lane);
  } else {
    acc.flush(a.slots + w, lane);
  }
}

// Sum and kept tokens of sequence s, by the `group` lanes of an aligned group
// (group a power of two up to 64): slots strided over the lanes, then a tree, so
// that the order depends on the sizes alone.
__device__ __forceinline__ void sequence_sum(const Seqs& q, const SeqPart* slots, int64_t s, int group, int lane,
                                             double& sum, int64_t& count) {
  int64_t b, e;   // slots [b, e)
  if (q.packed) {
    const int64_t t0 = load_offset(q, s), t1 = load_offset(q, s + 1);
    b = t0 / q.chunk + s;
    e = t1 > t0 ? (t1 - 1) / q.chunk + s + 1 : b;
  } else {
    b = s * q.chunks_per_row;
    e = b + q.chunks_per_row;
  }
  double x = 0.0;
  int64_t n = 0;
  for (int64_t i = b + (lane & (group - 1)); i < e; i += 4 * group) {
    SeqPart p[4];
#pragma unroll
    for (int j = 0; j < 4; j++) p[j] = slots[i + j * group < e ? i + j * group : i];   // four loads in flight
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (i + j * group < e) {
        x += p[j].sum;
        n += p[j].count;
      }
  }
  for (int o = 1; o < group; o <<= 1) {
    x += __shfl_xor(x, o);
    n += __shfl_xor(n, o);
  }
  sum = x;
  count = n;
}

// Sums of N values over the 1024 threads of a workgroup, in a fixed order; every thread gets them.
template <int N> __device__ __forceinline__ void block_sums(double (&x)[N], double (&lds)[16][4]) {
  static_assert(N <= 4, "");
  const int tid = threadIdx.x;
#pragma unroll
  for (int k = 0; k < N; k++) x[k] = wave_sum(x[k]);
  __syncthreads();
  if ((tid & 63) == 0)
#pragma unroll
    for (int k = 0; k < N; k++) lds[tid >> 6][k] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; k++) {
    x[k] = 0.0;
#pragma unroll
    for (int i = 0; i < 16; i++) x[k] += lds[i][k];
  }
}

// Per pair: the margin, its loss, and the factor its two sequences' tokens get in
// the gradient.  One workgroup: pairs are few next to tokens.
__global__ __launch_bounds__(1024) void preference_pairs_kernel(PreferenceArgs a) {
  __shared__ double lds[16][4];
  const int lane = lane_id();
  const int64_t P = a.q.S / 2;
  const int groups = 1024 / a.group, g = threadIdx.x / a.group;
  const bool lead = (threadIdx.x & (a.group - 1)) == 0;
  const double over_pairs = a.reduction == FLCE_REDUCTION_MEAN ? 1.0 / (double)(P > 0 ? P : 1) : 1.0;
  double total = 0.0;
  for (int64_t p0 = 0; p0 < P; p0 += groups) {   // whole waves stay in the loop: the sums exchange across lanes
    const int64_t p = p0 + g < P ? p0 + g : P - 1;
    double rc, rr;
    int64_t nc, nr;
    sequence_sum(a.q, a.slots, p, a.group, lane, rc, nc);
    sequence_sum(a.q, a.slots, P + p, a.group, lane, rr, nr);
    const double fc = a.normalize ? (nc > 0 ? 1.0 / (double)nc : 0.0) : 1.0;
    const double fr = a.normalize ? (nr > 0 ? 1.0 / (double)nr : 0.0) : 1.0;
    const double beta = a.beta;
    rc *= beta * fc;
    rr *= beta * fr;
    const double h = rc - rr - a.margin;
    double loss, slope;   // slope = d loss / d h
    if (a.type == FLCE_PREFERENCE_SIGMOID) {
      const double eps = a.smoothing;
      // -log sigmoid(h) = max(-h, 0) + near and -log sigmoid(-h) = max(h, 0) + near, each of one sign, and one
      // of weight 0 left out: an infinite margin is no inf - inf and no 0 times inf
      const double near = log1p(exp(-fabs(h)));
      loss = eps < 1.0 ? (1.0 - eps) * (fmax(-h, 0.0) + near) : 0.0;
      if (eps > 0.0) loss += eps * (fmax(h, 0.0) + near);
      slope = 1.0 / (1.0 + exp(-h)) - (1.0 - eps);
      if (eps == 0.0) slope = -1.0 / (1.0 + exp(h));
    } else if (a.type == FLCE_PREFERENCE_HINGE) {
      loss = h != h ? h : fmax(1.0 - h, 0.0);
      slope = h < 1.0 ? -1.0 : (h != h ? h : 0.0);
    } else {
      const double d = h / beta - 0.5 / beta;
      loss = d * d;
      slope = 2.0 * d / beta;
    }
    if (lead && p0 + g < P) {
      if (a.reduction == FLCE_REDUCTION_NONE) a.loss[p] = (float)loss;
      a.rewards[p] = (float)rc;
      a.rewards[P + p] = (float)rr;
      a.seq_grad[p] = (float)(slope * beta * fc * over_pairs);
      a.seq_grad[P + p] = (float)(-slope * beta * fr * over_pairs);
      total += loss;
    }
  }
  double all[1] = {total};
  block_sums(all, lds);
  if (threadIdx.x == 0 && a.reduction != FLCE_REDUCTION_NONE)
    a.loss[0] = a.reduction == FLCE_REDUCTION_MEAN && P == 0 ? __builtin_nanf("") : (float)(all[0] * over_pairs);
}

// The gradient of a token is its sequence's factor times the upstream value.
template <typename T, bool PACKED, bool VEC>
__global__ __launch_bounds__(256) void preference_grad_kernel(PreferenceGradArgs a) {
  const Seqs& q = a.q;
  const int lane = lane_id();
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= q.waves) return;
  const Chunk c = wave_chunk(q, w);
  const int64_t first = PACKED ? load_offset(q, 0) : 0, last = PACKED ? load_offset(q, q.S) : 0;
  const int64_t P = q.S / 2;
  const float g0 = a.per_pair ? 0.0f : a.grad_loss[0];
  SeqWalk walk;
  walk.s = 0;
  if (PACKED) walk.seek(q, c.begin, lane);
  T* out = reinterpret_cast<T*>(a.grad_logps) + c.row * q.length;
  uint32_t ahead = step_mask<VEC>(q, c, c.begin, step_size(c, c.begin), lane);
  for (int64_t t = c.begin; t < c.end; t += 256) {
    const int n = step_size(c, t);
    const uint32_t mask = ahead;
    ahead = step_mask<VEC>(q, c, t + 256, step_size(c, t + 256), lane);
    bool keep[4];
    int64_t seq[4];
    step_tokens<PACKED, VEC>(q, c, t, n, mask, true, walk, first, last, lane, keep, seq);
    float d[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      d[j] = 0.0f;
      if (keep[j]) {
        const float g = a.per_pair ? a.grad_loss[seq[j] < P ? seq[j] : seq[j] - P] : g0;
        d[j] = g * a.seq_grad[seq[j]];
      }
    }
    store_tokens<T, VEC>(out + t, n, lane, d);
  }
}

// ---------------------------------------------------------------------------
// Policy loss
// ---------------------------------------------------------------------------

// e^d - d - 1 >= 0.  Near 0 it is d^2 / 2: the difference of e^d - 1 and d would
// keep few of its digits there, so the series is summed instead (to d^9, a
// remainder below 2^-28 of the value for |d| <= 1/2).
__device__ __forceinline__ float exp_excess(float d, float em1) {
  if (d > 30.0f) return em1;   // d is below half a step of it (and may be infinite)
  if (fabsf(d) > 0.5f) return em1 - d;
  float s = fmaf(d, 1.0f / 362880.0f, 1.0f / 40320.0f);
  s = fmaf(d, s, 1.0f / 5040.0f);
  s = fmaf(d, s, 1.0f / 720.0f);
  s = fmaf(d, s, 1.0f / 120.0f);
  s = fmaf(d, s, 1.0f / 24.0f);
  s = fmaf(d, s, 1.0f / 6.0f);
  s = fmaf(d, s, 0.5f);
  return d * d * s;
}

template <typename T, bool PACKED, bool VEC>
__global__ __launch_bounds__(256) void policy_tokens_kernel(PolicyArgs a) {
  const Seqs& q = a.q;
  const int lane = lane_id();
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= q.waves) return;
  const Chunk c = wave_chunk(q, w);
  const int64_t first = PACKED ? load_offset(q, 0) : 0, last = PACKED ? load_offset(q, q.S) : 0;
  const bool sums = a.reduction == FLCE_REDUCTION_SEQUENCE_MEAN;   // a sum for each sequence, else one for the chunk
  const bool by_seq = PACKED && (sums || a.adv_per_seq);
  SeqWalk walk;
  walk.s = 0;
  if (by_seq) walk.seek(q, c.begin, lane);
  SeqSum acc;
  acc.clear();
  double kl = 0.0;
  int clipped = 0, kept = 0;
  const T* lp = reinterpret_cast<const T*>(a.logps) + c.row * a.ld_logps;
  const T* old = reinterpret_cast<const T*>(a.old) + c.row * a.ld_old;
  const T* ref = a.ref ? reinterpret_cast<const T*>(a.ref) + c.row * a.ld_ref : nullptr;
  const bool with_ent = a.entropy && a.entropy_coef != 0.0f;   // (0 times what entropies hold may be NaN)
  const T* ent = with_ent ? reinterpret_cast<const T*>(a.entropy) + c.row * a.ld_entropy : nullptr;
  const float* adv = a.adv_per_seq ? a.adv : a.adv + c.row * a.ld_adv;
  auto load = [&](int64_t t, StepIn<5>& in) {
    const int n = step_size(c, t);
    load_tokens<T, VEC>(lp + t, n, lane, in.x[0]);
    load_tokens<T, VEC>(old + t, n, lane, in.x[1]);
    if (!a.adv_per_seq) load_tokens<float, VEC>(adv + t, n, lane, in.x[2]);
    if (ref) load_tokens<T, VEC>(ref + t, n, lane, in.x[3]);
    if (ent) load_tokens<T, VEC>(ent + t, n, lane, in.x[4]);
    in.mask = step_mask<VEC>(q, c, t, n, lane);
  };
  StepIn<5> in, ahead;
  load(c.begin, in);
  for (int64_t t = c.begin; t < c.end; t += 256, in = ahead) {
    load(t + 256, ahead);
    const int n = step_size(c, t);
    const float(&x)[4] = in.x[0], (&o)[4] = in.x[1], (&A)[4] = in.x[2], (&r)[4] = in.x[3], (&h)[4] = in.x[4];
    bool keep[4];
    int64_t seq[4];
    const int64_t from = walk.s;
    step_tokens<PACKED, VEC>(q, c, t, n, in.mask, by_seq, walk, first, last, lane, keep, seq);
    if (a.adv_per_seq) {
#pragma unroll
      for (int j = 0; j < 4; j++) in.x[2][j] = keep[j] ? adv[seq[j]] : 0.0f;
    }
    float loss[4], grad[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      // the side of a border in fp64: logp - old rounded to fp32 would move
      // tokens across it, and their gradient is then all or nothing
      const double xd = (double)x[j] - (double)o[j];
      const float ratio = expf((float)xd);
      const bool neg = A[j] < 0.0f;
      bool active = A[j] == 0.0f || (neg ? !(xd < a.log_low) : !(xd > a.log_high));
      const float plain = A[j] == 0.0f ? 0.0f : ratio * A[j];   // an overflowed ratio times no advantage is 0
      float gain = active ? plain : (neg ? a.low : a.high) * A[j];
      if (a.dual > 0.0f && neg && xd > a.log_dual) {
        gain = a.dual * A[j];
        active = false;
      }
      float l = -gain, d = active ? -plain : 0.0f;
      if (ref) {
        const float away = r[j] - x[j], em1 = expm1f(away);
        const float k = exp_excess(away, em1);
        if (a.kl_coef != 0.0f) {   // (0 times an infinite k, of a reference for its metric alone, is NaN)
          l = fmaf(a.kl_coef, k, l);
          d = fmaf(-a.kl_coef, em1, d);
        }
        if (keep[j]) kl += (double)k;
      }
      if (ent) l = fmaf(-a.entropy_coef, h[j], l);
      loss[j] = keep[j] ? l : 0.0f;
      grad[j] = keep[j] ? d : 0.0f;
      if (keep[j]) {
        clipped += active ? 0 : 1;
        kept++;
      }
    }
    if (a.unit_grad) store_tokens<float, VEC>(a.unit_grad + c.row * q.length + t, n, lane, grad);
    if (a.reduction == FLCE_REDUCTION_NONE) store_tokens<float, VEC>(a.loss + c.row * q.length + t, n, lane, loss);
    acc.add(q, a.slots, w, sums ? from : 0, sums && PACKED ? walk.s : (sums ? from : 0), keep, seq, loss, lane);
  }
  if (PACKED && sums) {
    if (walk.s >= 0 && walk.s < q.S) acc.flush(a.slots + w + walk.s, lane);
  } else {
    acc.flush(a.slots + w, lane);
  }
  kl = wave_sum(kl);
  clipped = wave_sum(clipped);
  kept = wave_sum(kept);
  if (lane == 0) {
    WavePart m;
    m.kl = kl;
    m.clipped = clipped;
    m.kept = kept;
    a.parts[w] = m;
  }
}

// The sum or mean, the weights of the tokens' losses in it, and the metrics.
__global__ __launch_bounds__(1024) void policy_merge_kernel(PolicyArgs a) {
  __shared__ double lds[16][4];
  const int tid = threadIdx.x, lane = lane_id();
  const Seqs& q = a.q;
  double kl = 0.0, clipped = 0.0, kept = 0.0, total = 0.0, filled = 0.0;
  const bool sums = a.reduction == FLCE_REDUCTION_SEQUENCE_MEAN;
  for (int64_t w = tid; w < q.waves; w += 1024) {
    kl += a.parts[w].kl;
    clipped += (double)a.parts[w].clipped;
    kept += (double)a.parts[w].kept;
    if (!sums) total += a.slots[w].sum;
  }
  if (sums) {
    const int groups = 1024 / a.group, g = tid / a.group;
    const bool lead = (tid & (a.group - 1)) == 0;
    for (int64_t s0 = 0; s0 < q.S; s0 += groups) {   // whole waves stay in the loop
      const int64_t s = s0 + g < q.S ? s0 + g : q.S - 1;
      double x;
      int64_t n;
      sequence_sum(q, a.slots, s, a.group, lane, x, n);
      if (lead && s0 + g < q.S) {
        if (n > 0) {
          total += x / (double)n;
          filled += 1.0;
        }
        // the number of sequences is known only after this loop: weights[0] holds its factor
        a.weights[1 + s] = n > 0 ? (float)(1.0 / (double)n) : 0.0f;
      }
    }
  }
  double all[4] = {kl, clipped, kept, total};
  block_sums(all, lds);
  kl = all[0];
  clipped = all[1];
  kept = all[2];
  total = all[3];
  double weight = 1.0;
  if (sums) {
    double f[1] = {filled};
    block_sums(f, lds);
    weight = f[0] > 0.0 ? 1.0 / f[0] : 0.0;
  } else if (a.reduction == FLCE_REDUCTION_MEAN) {
    weight = kept > 0.0 ? 1.0 / kept : 0.0;
  }
  if (tid == 0) {
    a.weights[0] = (float)weight;
    if (a.reduction != FLCE_REDUCTION_NONE) a.loss[0] = weight > 0.0 ? (float)(total * weight) : __builtin_nanf("");
    if (a.metrics) {
      a.metrics->num_tokens = (int64_t)kept;
      a.metrics->clip_fraction = (float)(clipped / kept);
      a.metrics->kl = (float)(kl / kept);
    }
  }
}

template <typename T, bool PACKED, bool VEC>
__global__ __launch_bounds__(256) void policy_grad_kernel(PolicyGradArgs a) {
  const Seqs& q = a.q;
  const int lane = lane_id();
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= q.waves) return;
  const Chunk c = wave_chunk(q, w);
  const int64_t first = PACKED ? load_offset(q, 0) : 0, last = PACKED ? load_offset(q, q.S) : 0;
  const bool by_seq = PACKED && a.seq_weights;
  const float g0 = (a.per_token ? 1.0f : a.grad_loss[0]) * a.weights[0];
  SeqWalk walk;
  walk.s = 0;
  if (by_seq) walk.seek(q, c.begin, lane);
  const int64_t row = c.row * q.length;
  auto load = [&](int64_t t, StepIn<2>& in) {
    const int n = step_size(c, t);
    if (a.grad_logps) load_tokens<float, VEC>(a.unit_grad + row + t, n, lane, in.x[0]);
    if (a.per_token) load_tokens<float, VEC>(a.grad_loss + row + t, n, lane, in.x[1]);
    in.mask = step_mask<VEC>(q, c, t, n, lane);
  };
  StepIn<2> in, ahead;
  load(c.begin, in);
  for (int64_t t = c.begin; t < c.end; t += 256, in = ahead) {
    load(t + 256, ahead);
    const int n = step_size(c, t);
    bool keep[4];
    int64_t seq[4];
    step_tokens<PACKED, VEC>(q, c, t, n, in.mask, by_seq, walk, first, last, lane, keep, seq);
    float d[4], e[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float g = a.per_token ? in.x[1][j] * g0 : g0;
      if (a.seq_weights) g *= keep[j] ? a.weights[1 + seq[j]] : 0.0f;
      d[j] = keep[j] && a.grad_logps ? g * in.x[0][j] : 0.0f;
      e[j] = keep[j] ? g * -a.entropy_coef : 0.0f;
    }
    if (a.grad_logps) store_tokens<T, VEC>(reinterpret_cast<T*>(a.grad_logps) + row + t, n, lane, d);
    if (a.grad_entropy) store_tokens<T, VEC>(reinterpret_cast<T*>(a.grad_entropy) + row + t, n, lane, e);
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <typename F> static void by_layout(int dtype, bool packed, bool vec, F f) {
  auto with = [&](auto t) {
    using T = decltype(t);
    if (packed) {
      if (vec) f.template run<T, true, true>();
      else f.template run<T, true, false>();
    } else {
      if (vec) f.template run<T, false, true>();
      else f.template run<T, false, false>();
    }
  };
  if (dtype == FLCE_BF16) with(bf16());
  else if (dtype == FLCE_F16) with(f16());
  else with(0.0f);
}

static unsigned wave_blocks(const Seqs& q) { return (unsigned)((q.waves + 3) / 4); }

struct RunPreference {
  const PreferenceArgs& a;
  hipStream_t st;
  template <typename T, bool P, bool V> void run() const {
    preference_tokens_kernel<T, P, V><<<wave_blocks(a.q), 256, 0, st>>>(a);
  }
};
struct RunPreferenceGrad {
  const PreferenceGradArgs& a;
  hipStream_t st;
  template <typename T, bool P, bool V> void run() const {
    preference_grad_kernel<T, P, V><<<wave_blocks(a.q), 256, 0, st>>>(a);
  }
};
struct RunPolicy {
  const PolicyArgs& a;
  hipStream_t st;
  template <typename T, bool P, bool V> void run() const {
    policy_tokens_kernel<T, P, V><<<wave_blocks(a.q), 256, 0, st>>>(a);
  }
};
struct RunPolicyGrad {
  const PolicyGradArgs& a;
  hipStream_t st;
  template <typename T, bool P, bool V> void run() const {
    policy_grad_kernel<T, P, V><<<wave_blocks(a.q), 256, 0, st>>>(a);
  }
};

hipError_t launch_preference(int dtype, bool vec, const PreferenceArgs& a, hipStream_t st) {
  if (a.q.waves > 0) by_layout(dtype, a.q.packed != 0, vec, RunPreference{a, st});
  preference_pairs_kernel<<<1, 1024, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_preference_grad(int dtype, bool vec, const PreferenceGradArgs& a, hipStream_t st) {
  if (a.q.waves > 0) by_layout(dtype, a.q.packed != 0, vec, RunPreferenceGrad{a, st});
  return hipGetLastError();
}

hipError_t launch_policy(int dtype, bool vec, const PolicyArgs& a, hipStream_t st) {
  if (a.q.waves > 0) by_layout(dtype, a.q.packed != 0, vec, RunPolicy{a, st});
  policy_merge_kernel<<<1, 1024, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_policy_grad(int dtype, bool vec, const PolicyGradArgs& a, hipStream_t st) {
  if (a.q.waves > 0) by_layout(dtype, a.q.packed != 0, vec, RunPolicyGrad{a, st});
  return hipGetLastError();
}

}  // namespace flce
