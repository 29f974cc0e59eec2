// Per-token log-probabilities and entropies of a linear head, without its logits:
// the tile loop of the forward pass with an epilogue of its own, then a merge of
// the vocabulary splits.
//
// Everything is kept in base 2: y = z log2(e), so that an exponential is one
// v_exp and the running maximum, sums and target need no conversions.  Per row,
// over the logits seen so far,
//   m = max y,   l = sum 2^(y - m),   T = sum 2^(y - m) (y - m),
// and at the end  log2 p_t = y_t - m - log2 l,  H = ln 2 (log2 l - T / l).
// T is taken relative to the maximum: H = lse - sum p z would subtract two numbers
// of the size of the logits, and a near-certain row's small entropy would be lost
// in their rounding; log2 l and T / l both go to 0 there.  On a new maximum m' =
// m + d, l' = l 2^-d and T' = (T - d l) 2^-d.
//
// With 8-bit operands (a frozen scorer's head) the accumulator is the exact int32
// product; one multiplication by the vocabulary row's scale and one by the token's
// turn it into the logit, and the rest is the same.
#include <math.h>

#include "flce_device.h"
#include "flce_logprobs.h"
#include "flce_lp_state.h"

namespace flce {

template <typename T, bool HAS_BIAS, bool SOFTCAP>
__global__ __launch_bounds__(kThreads, 1) void lp_tiles_kernel(LpTileArgs a) {
  constexpr int E = sizeof(T);
  constexpr bool I8 = E == 1;
  typedef typename BiasOf<T>::type B;
  constexpr int BE = sizeof(B);
  const int L = xcd_logical_id(blockIdx.x, gridDim.x);
  // the tile order of fwd_tiles_kernel: 4 token tiles x 8 splits on an XCD at a time
  const int n_tt = (int)gridDim.x / a.S;
  const bool grouped = a.S % 8 == 0 && n_tt % 4 == 0 && gridDim.x >= 256;
  int tt, s;
  if (grouped) {
    grouped_tile(L, n_tt, a.S, 4, tt, s);
  } else {
    tt = L / a.S;
    s = L % a.S;
  }
  const int vt_begin = (int)((int64_t)s * a.n_vt / a.S);
  const int vt_end = (int)((int64_t)(s + 1) * a.n_vt / a.S);
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const int t0 = tt * 256;
  if (blockIdx.x == 0 && tid == 0) a.status[0] = FLCE_OK;

  // m and l in registers, T, the target's logit and the targets in LDS, where they
  // wait out the main loop
  static __shared__ float st_T[kWaves][kNI][64], st_yt[kWaves][kNI][64];
  static __shared__ int tile_tgt[256];
  static __shared__ float tile_scale[I8 ? 256 : 1];   // the tokens' scales
  float st_m[kNI], st_l[kNI];
#pragma unroll
  for (int ni = 0; ni < kNI; ni++) {
    st_m[ni] = kMasked;
    st_l[ni] = 0.0f;
    st_T[wave][ni][lane] = 0.0f;
    st_yt[wave][ni][lane] = -INFINITY;
  }
  if (tid < 256) {   // visible to all waves after the main loop's first barrier
    const int t = t0 + tid;
    const int64_t tv = t < a.N ? load_target(a.targets, t, a.tgt_i32) : a.ignore_index;
    tile_tgt[tid] = (tv != a.ignore_index && tv >= 0 && tv < a.V) ? (int)tv : -1;
    if (I8) tile_scale[tid] = t < a.N ? a.hidden_scale[t] : 0.0f;
  }

  const uint32_t ld = (uint32_t)a.H * E;
  OperandDesc db;     // hidden rows of this token tile
  db.base = a.hidden + (size_t)t0 * ld;
  db.ld_bytes = ld;
  db.nrec = (uint32_t)min(a.N - t0, 256) * ld;
  db.cols_valid = 0;
  db.k_bytes = a.H * E;
  const int KT = (a.H * E + kBKB - 1) / kBKB;

  const int win = min(32, max(1, (int)gridDim.x / 8));
  L2Share sh;
  if (grouped) {
    sh.a_n = 4;
    sh.a_rank = tt & 3;
    sh.b_n = 8;
    sh.b_rank = s & 7;
  } else {
    sh.b_n = min(a.S, win);
    sh.b_rank = s % sh.b_n;
    sh.a_n = a.S <= win ? win / a.S : 1;
    sh.a_rank = tt % sh.a_n;
    if (sh.a_n < 2) sh.a_n = 0;
    if (sh.b_n < 2) sh.b_n = 0;
  }

  // two buffers, by tile parity (see fwd_tiles_kernel)
  static __shared__ __attribute__((aligned(16))) char bias_lds[2][256 * BE], wscale_lds[2][I8 ? 1024 : 16];

  // the accumulator times s_u is u = y, or with the cap u = v / cap, y = cap log2(e) tanh(u).
  // (N = 8192, H = 4096, V = 32768, cap 30: bf16 1570 us with all logits below 24, 1618 with most
  // above; 8-bit 887, 940.  1 - 2 / (e^2u + 1) for all, off by 1e-7 of the cap: 1548, 865.)
  const float s_u = SOFTCAP ? a.scale / a.cap : a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e;
  auto capped = [&](float u) { return cap2 * tanh_of<true>(u); };

  Acc acc[kMI][kNI];
  for (int vt = vt_begin; vt < vt_end; ++vt) {
    const int v0 = a.v_first + vt * 256;
    const char* bias_tile = bias_lds[(vt - vt_begin) & 1];
    if (HAS_BIAS && wave == 0)
      dma_vector(reinterpret_cast<const B*>(a.bias) + v0, ((uint32_t)min(a.V - v0, 256) * BE + 3u) & ~3u,
                 bias_lds[(vt - vt_begin) & 1], 256 * BE, lane);
    if (I8 && wave == 1)
      dma_vector(a.weight_scale + v0, (uint32_t)min(a.V - v0, 256) * 4, wscale_lds[(vt - vt_begin) & 1], 1024, lane);
    OperandDesc da;     // weight rows of this vocabulary tile
    da.base = a.weight + (size_t)v0 * ld;
    da.ld_bytes = ld;
    da.nrec = (uint32_t)min(a.V - v0, 256) * ld;
    da.cols_valid = 0;
    da.k_bytes = a.H * E;
    zero_acc(acc);
    tile_mainloop<T, true, true>(da, db, KT, sh, acc);

    // per token column: pass 1 turns the accumulator into u and takes the maximum
    // over the rows below V, pass 2 adds 2^x and x 2^x, x = y - m <= 0
    const int vw = v0 + wm * kWaveM;
    const int n_valid = a.V - vw;
    const bool ragged = n_valid < kWaveM;
    const int lane_row = acc_row(0, 0, lane);
    const int lim = n_valid - lane_row;   // element (mi, r) is below V iff 16 mi + r < lim
    if constexpr (I8) {
#pragma unroll
      for (int mi = 0; mi < kMI; mi++) {
        const f32x4 ws =
            *reinterpret_cast<const f32x4*>(wscale_lds[(vt - vt_begin) & 1] + 4 * (wm * kWaveM + acc_row(mi, 0, lane)));
#pragma unroll
        for (int ni = 0; ni < kNI; ni++)
#pragma unroll
          for (int r = 0; r < 4; r++) acc[mi][ni][r] = (float)__builtin_bit_cast(int, (float)acc[mi][ni][r]) * ws[r];
      }
    }
#pragma unroll
    for (int ni = 0; ni < kNI; ni++) {
      const float s_a = I8 ? s_u * tile_scale[wn * kWaveN + acc_col(ni, lane)] : s_u;
      float mu = kMasked;
#pragma unroll
      for (int mi = 0; mi < kMI; mi++) {
        float sb[4];
        if constexpr (HAS_BIAS) {
          lds_vec4<B>(bias_tile, wm * kWaveM + acc_row(mi, 0, lane), sb);
#pragma unroll
          for (int j = 0; j < 4; j++) sb[j] *= s_u;
        }
#pragma unroll
        for (int r = 0; r < 4; r++)
          acc[mi][ni][r] = HAS_BIAS ? fmaf(acc[mi][ni][r], s_a, sb[r]) : acc[mi][ni][r] * s_a;
      }
      if (ragged) {
#pragma unroll
        for (int mi = 0; mi < kMI; mi++)
#pragma unroll
          for (int r = 0; r < 4; r++)
            if (16 * mi + r < lim) mu = fmaxf(mu, acc[mi][ni][r]);
      } else {
#pragma unroll
        for (int mi = 0; mi < kMI; mi++)
#pragma unroll
          for (int r = 0; r < 4; r++) mu = fmaxf(mu, acc[mi][ni][r]);
      }
      // a block without a finite logit keeps kMasked, with the cap one without a row (there a
      // logit of -inf is -cap)
      const float mx = SOFTCAP && lim > 0 ? capped(mu) : mu;
      const int rel = tile_tgt[wn * kWaveN + acc_col(ni, lane)] - vw;
      const bool hit = rel >= 0 && rel < kWaveM && ((rel >> 2) & 3) == (lane >> 4);
      if (__builtin_amdgcn_ballot_w64(hit)) {
        const int rel_l = rel - lane_row;
        float ut = 0.0f;
#pragma unroll
        for (int mi = 0; mi < kMI; mi++)
#pragma unroll
          for (int r = 0; r < 4; r++)
            if (16 * mi + r == rel_l) ut = acc[mi][ni][r];
        if (hit) st_yt[wave][ni][lane] = SOFTCAP ? capped(ut) : ut;
      }
      const float m_old = st_m[ni];
      const float m_new = fmaxf(m_old, mx);
      const float dm = st_l[ni] == 0.0f ? 0.0f : m_old - m_new;
      const float alpha = fast_exp2(dm);
      float se0 = 0.f, se1 = 0.f, sx0 = 0.f, sx1 = 0.f;
#pragma unroll
      for (int mi = 0; mi < kMI; mi++) {
        float u[4], th[4];
#pragma unroll
        for (int r = 0; r < 4; r++) u[r] = acc[mi][ni][r];
        if constexpr (SOFTCAP) tanh4(u, th);
#pragma unroll
        for (int r = 0; r < 4; r++) {
          float x = SOFTCAP ? fmaf(cap2, th[r], -m_new) : u[r] - m_new;
          if (ragged && 16 * mi + r >= lim) x = kMasked;
          const float e = fast_exp2(x);
          // a logit of -inf (there is none with the cap, nor of 8-bit products without a
          // bias) has e = 0 and is to add 0, not 0 times infinity
          const float xf = SOFTCAP || (I8 && !HAS_BIAS) ? x : fmaxf(x, kMasked);
          if (r & 1) {
            se1 += e;
            sx1 = fmaf(e, xf, sx1);
          } else {
            se0 += e;
            sx0 = fmaf(e, xf, sx0);
          }
        }
      }
      st_T[wave][ni][lane] = fmaf(fmaf(dm, st_l[ni], st_T[wave][ni][lane]), alpha, sx0 + sx1);
      st_l[ni] = fmaf(st_l[ni], alpha, se0 + se1);
      st_m[ni] = m_new;
    }
  }

  LpState st[kNI];
#pragma unroll
  for (int ni = 0; ni < kNI; ni++) {
    st[ni].m = st_m[ni];
    st[ni].l = st_l[ni];
    st[ni].T = st_T[wave][ni][lane];
    st[ni].yt = st_yt[wave][ni][lane];
  }
  // the four lanes of a token column hold disjoint rows
#pragma unroll
  for (int ni = 0; ni < kNI; ni++) {
#pragma unroll
    for (int x = 16; x <= 32; x <<= 1) {
      LpState o;
      o.m = __shfl_xor(st[ni].m, x);
      o.l = __shfl_xor(st[ni].l, x);
      o.T = __shfl_xor(st[ni].T, x);
      o.yt = __shfl_xor(st[ni].yt, x);
      lp_merge(st[ni], o);
    }
  }
  // the two M waves, through LDS
  static_assert(kWavesM == 2, "the merge below pairs two waves along M");
  float* xs = reinterpret_cast<float*>(g_stage0);   // [wn][field][kWaveN]
  if (wm == 1 && lane < 16) {
#pragma unroll
    for (int ni = 0; ni < kNI; ni++) {
      float* p = xs + wn * 4 * kWaveN + acc_col(ni, lane);
      p[0 * kWaveN] = st[ni].m;
      p[1 * kWaveN] = st[ni].l;
      p[2 * kWaveN] = st[ni].T;
      p[3 * kWaveN] = st[ni].yt;
    }
  }
  __syncthreads();
  if (wm == 0 && lane < 16) {
    const size_t plane = (size_t)a.S_all * a.N_pad;
#pragma unroll
    for (int ni = 0; ni < kNI; ni++) {
      const int c = acc_col(ni, lane);
      const float* p = xs + wn * 4 * kWaveN + c;
      LpState o;
      o.m = p[0 * kWaveN];
      o.l = p[1 * kWaveN];
      o.T = p[2 * kWaveN];
      o.yt = p[3 * kWaveN];
      lp_merge(st[ni], o);
      float* out = a.part + (size_t)(a.s_first + s) * a.N_pad + t0 + wn * kWaveN + c;
      out[0] = st[ni].m;
      out[plane] = st[ni].l;
      out[2 * plane] = st[ni].T;
      out[3 * plane] = st[ni].yt;
    }
  }
}

// Merges each row's vocabulary splits and writes its outputs.  A workgroup takes 16 rows
// by `subs` threads each (a power of two from 4 to 64), neighbouring threads on
// neighbouring rows; a thread merges every subs-th split, then lanes, then waves merge,
// all in an order that depends on the sizes alone.  (Few rows have hundreds of splits:
// one thread to a row took 38 us for 4 rows of 256.)
struct LpRowArgs {
  const void* targets;
  int tgt_i32;
  int N, V, S, N_pad, subs;
  int64_t ignore_index;
  const float* part;
  float* logps;
  float* entropy;   // may be NULL
  float* lse;
  int* status;
  int init_status;  // no tile kernel ran before (N = 0)
};

__device__ __forceinline__ LpState lp_lane_merge(LpState r) {   // over lanes l, l ^ 16, l ^ 32, l ^ 48
#pragma unroll
  for (int o = 16; o <= 32; o <<= 1) {
    LpState q;
    q.m = __shfl_xor(r.m, o);
    q.l = __shfl_xor(r.l, o);
    q.T = __shfl_xor(r.T, o);
    q.yt = __shfl_xor(r.yt, o);
    lp_merge(r, q);
  }
  return r;
}

__global__ __launch_bounds__(1024) void lp_rows_kernel(LpRowArgs a) {
  __shared__ LpState waves[16][16];
  const int tid = threadIdx.x, sub = tid >> 4, i = (int)blockIdx.x * 16 + (tid & 15);
  if (a.init_status && blockIdx.x == 0 && tid == 0) a.status[0] = FLCE_OK;
  if (a.N == 0) return;
  const int row = min(i, a.N - 1);   // threads past the last row stay in step
  const size_t plane = (size_t)a.S * a.N_pad;
  const int64_t t = load_target(a.targets, row, a.tgt_i32);
  LpState r{kMasked, 0.0f, 0.0f, -INFINITY};
  for (int s0 = sub; s0 < a.S; s0 += 4 * a.subs) {
    LpState q[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {   // four splits' loads in flight; past the last one it again, not merged
      const float* p = a.part + (size_t)min(s0 + j * a.subs, a.S - 1) * a.N_pad + row;
      q[j].m = p[0];
      q[j].l = p[plane];
      q[j].T = p[2 * plane];
      q[j].yt = p[3 * plane];
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (s0 + j * a.subs < a.S) lp_merge(r, q[j]);
  }
  r = lp_lane_merge(r);
  const int n_waves = a.subs >> 2;
  if (n_waves > 1) {
    if ((tid & 63) < 16) waves[tid >> 6][tid & 15] = r;
    __syncthreads();
    if (tid >= 64) return;
    r = LpState{kMasked, 0.0f, 0.0f, -INFINITY};
    for (int w = sub; w < n_waves; w += 4) lp_merge(r, waves[w][tid & 15]);
    r = lp_lane_merge(r);
  }
  if (sub != 0 || i >= a.N) return;
  const float l2 = fast_log2(r.l);
  const bool in_range = t >= 0 && t < a.V, valid = t != a.ignore_index && in_range;
  // (a row without any finite logit: l = 0, and every output is NaN or -inf)
  a.lse[i] = (r.m + l2) * kLn2;
  a.logps[i] = valid ? (r.yt - r.m - l2) * kLn2 : 0.0f;
  if (a.entropy) a.entropy[i] = valid ? (l2 - r.T / r.l) * kLn2 : 0.0f;
  if (t != a.ignore_index && !in_range) a.status[0] = FLCE_ERR_TARGET_OUT_OF_RANGE;   // every writer stores the same
}

template <typename T>
static void launch_lp_tiles(const Plan& pl, const LpTileArgs& a, int nwg, hipStream_t st) {
  if (pl.has_bias) {
    if (pl.cap > 0) lp_tiles_kernel<T, true, true><<<nwg, kThreads, 0, st>>>(a);
    else lp_tiles_kernel<T, true, false><<<nwg, kThreads, 0, st>>>(a);
  } else {
    if (pl.cap > 0) lp_tiles_kernel<T, false, true><<<nwg, kThreads, 0, st>>>(a);
    else lp_tiles_kernel<T, false, false><<<nwg, kThreads, 0, st>>>(a);
  }
}

// ---------------------------------------------------------------------------
// Rows as 8-bit integers: s = max|x| / 127 and q = rint(x / s), in fp32 as
// s = max|x| * fp32(1/127), q = rint(x * fp32(1/s)), so that every implementation
// of the definition gives the same integers.  A row that is (nearly) all zero has
// s = 0 and q = 0; a row that holds NaN or an infinity has s = NaN and q = 0.  One
// workgroup a row; the second pass reads the row from cache.
// ---------------------------------------------------------------------------
constexpr float kQuantTiny = 1e-30f;   // 1 / s stays finite above it

template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int64_t cols, int8_t* q, float* scale) {
  __shared__ float lds[4];
  const int tid = threadIdx.x;
  const T* row = x + (int64_t)blockIdx.x * cols;
  int8_t* out = q + (int64_t)blockIdx.x * cols;
  constexpr int kVec = 16 / sizeof(T);
  typedef T TV __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef int8_t QV __attribute__((ext_vector_type(16 / sizeof(T))));
  const int64_t n = cols / kVec;
  float top = 0.0f;
  bool bad = false;
  for (int64_t i = tid; i < n; i += 256) {
    const TV v = reinterpret_cast<const TV*>(row)[i];
#pragma unroll
    for (int j = 0; j < kVec; j++) {
      const float f = fabsf((float)v[j]);
      top = fmaxf(top, f);
      bad = bad || !(f < INFINITY);
    }
  }
  if (bad) top = INFINITY;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if ((tid & 63) == 0) lds[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
  const bool zero = !(top >= kQuantTiny && top < INFINITY);
  const float s = top * (1.0f / 127.0f), r = zero ? 0.0f : 1.0f / s;
  if (tid == 0) scale[blockIdx.x] = top == INFINITY ? __builtin_nanf("") : (zero ? 0.0f : s);
  for (int64_t i = tid; i < n; i += 256) {
    const TV v = reinterpret_cast<const TV*>(row)[i];
    QV o;
#pragma unroll
    for (int j = 0; j < kVec; j++) {
      const float f = zero ? 0.0f : rintf((float)v[j] * r);
      o[j] = (int8_t)(int)fminf(fmaxf(f, -127.0f), 127.0f);
    }
    reinterpret_cast<QV*>(out)[i] = o;
  }
}

template <typename T>
static void launch_quantize_t(const void* x, int64_t rows, int64_t cols, int8_t* q, float* scale, hipStream_t st) {
  constexpr int64_t kMost = int64_t(1) << 22;   // a launch of 2^32 threads or more leaves workgroups out
  for (int64_t r = 0; r < rows; r += kMost)
    quantize_rows_kernel<T><<<(unsigned)(rows - r < kMost ? rows - r : kMost), 256, 0, st>>>(
        static_cast<const T*>(x) + r * cols, cols, q + r * cols, scale + r);
}

hipError_t launch_quantize(int dtype, const void* x, int64_t rows, int64_t cols, int8_t* q, float* scale,
                           hipStream_t st) {
  if (dtype == FLCE_BF16) launch_quantize_t<bf16>(x, rows, cols, q, scale, st);
  else if (dtype == FLCE_F16) launch_quantize_t<f16>(x, rows, cols, q, scale, st);
  else launch_quantize_t<float>(x, rows, cols, q, scale, st);
  return hipGetLastError();
}

hipError_t launch_logprobs(const Plan& pl, const LpPlan& lp, const void* hidden, const void* weight, const void* bias,
                           const float* hidden_scale, const float* weight_scale, const void* targets, float* logps,
                           float* entropy, float* lse, char* ws, hipStream_t st) {
  float* part = reinterpret_cast<float*>(ws + kStatusBytes);
  int* status = reinterpret_cast<int*>(ws);
  if (pl.N > 0) {
    LpTileArgs a;
    a.hidden = static_cast<const char*>(hidden);
    a.weight = static_cast<const char*>(weight);
    a.bias = bias;
    a.hidden_scale = hidden_scale;
    a.weight_scale = weight_scale;
    a.targets = targets;
    a.tgt_i32 = pl.tgt_i32 ? 1 : 0;
    a.N = (int)pl.N;
    a.H = (int)pl.H;
    a.V = (int)pl.V;
    a.ignore_index = pl.ignore_index;
    a.scale = pl.scale;
    a.cap = pl.cap;
    a.S_all = lp.S_large + lp.S_small;
    a.N_pad = lp.N_pad;
    a.part = part;
    a.status = status;
    if (lp.vt_large > 0) {
      a.v_first = 0;
      a.n_vt = lp.vt_large;
      a.S = lp.S_large;
      a.s_first = 0;
      const int nwg = (int)pl.n_tt * a.S;
      if (pl.int8) launch_lp_tiles<int8_t>(pl, a, nwg, st);
      else if (pl.dtype == FLCE_BF16) launch_lp_tiles<bf16>(pl, a, nwg, st);
      else if (pl.dtype == FLCE_F16) launch_lp_tiles<f16>(pl, a, nwg, st);
      else launch_lp_tiles<float>(pl, a, nwg, st);
    }
    if (lp.S_small > 0) {
      a.v_first = lp.vt_large * 256;
      a.n_vt = (a.V - a.v_first + 63) / 64;
      a.S = lp.S_small;
      a.s_first = lp.S_large;
      launch_lp_small(pl, lp.bn, a, (a.N + lp.bn - 1) / lp.bn, st);
    }
  }
  LpRowArgs r;
  r.targets = targets;
  r.tgt_i32 = pl.tgt_i32 ? 1 : 0;
  r.N = (int)pl.N;
  r.V = (int)pl.V;
  r.S = lp.S_large + lp.S_small;
  r.N_pad = lp.N_pad;
  r.subs = 4;
  while (r.subs < 64 && r.subs < r.S) r.subs *= 2;
  r.ignore_index = pl.ignore_index;
  r.part = part;
  r.logps = logps;
  r.entropy = entropy;
  r.lse = lse;
  r.status = status;
  r.init_status = pl.N == 0;
  const int64_t blocks = (pl.N + 15) / 16;
  lp_rows_kernel<<<(unsigned)(blocks > 0 ? blocks : 1), 16 * r.subs, 0, st>>>(r);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Backward: the loss's, with these per-row constants.
// ---------------------------------------------------------------------------
// With upstream gradients
// g of log p_t and h of H,
//   d / d z_j = g [j = t] - p_j (g + h (H + log p_j))
//             = coefA p_j + coefE p_j log2 p_j - coefB [j = t],
// coefA = -(g + h H), coefE = -h ln 2, coefB = -g.  The kernels subtract the LSE in base 2,
// L, as one fp32 number.  The saved LSE is in nats; the rounding of its conversion to base 2
// (1e-6 at 16 to 32, which every p of the row would carry) is taken back by the constants:
// with L = Lf + d and p = 2^-d p',
//   coefA p + coefE p log2 p = p' (2^-d (coefA - d coefE) + 2^-d coefE log2 p').
// What stays in every p of a row are the forward's own roundings, of m + log2 l and of its
// product with ln 2.
struct LpPrepArgs {
  const void* targets;
  int tgt_i32;
  const float* lse;
  const float* entropy;
  const float* grad_logps;
  const float* grad_entropy;
  int N, V, N_pad;
  int64_t ignore_index;
  float* coefA;
  float* coefB;
  float* coefE;
  float* lseL;
  int* tgt;
  int* status;
  float* dscale;
  int f16_d;
  float abs_scale;
};

__global__ __launch_bounds__(1024) void lp_prep_kernel(LpPrepArgs a) {
  __shared__ float sm[1024];
  __shared__ int sb[1024];
  const int tid = threadIdx.x;
  float dmax = 0.0f;
  int bad = 0;
  for (int i = tid; i < a.N_pad; i += 1024) {
    // padding and ignored rows: coefficients 0 and an LSE beyond any logit, so that p = 0,
    // but finite, so that coefE log2 p is 0 too
    float ca = 0.0f, cb = 0.0f, ce = 0.0f, ll = -kMasked;
    int tg = -1;
    if (i < a.N) {
      const int64_t t = load_target(a.targets, i, a.tgt_i32);
      const bool in_range = t >= 0 && t < a.V;
      bad |= (t != a.ignore_index && !in_range) ? 1 : 0;
      if (t != a.ignore_index && in_range) {
        const double exact = (double)a.lse[i] / (double)kLn2;   // the constant that lp_rows_kernel multiplied by
        ll = (float)exact;
        const float d = fabsf(ll) < INFINITY ? (float)(exact - (double)ll) : 0.0f;
        const float g = a.grad_logps ? a.grad_logps[i] : 0.0f;
        const float h = a.grad_entropy ? a.grad_entropy[i] : 0.0f;
        cb = -g;
        ca = a.grad_entropy ? -fmaf(h, a.entropy[i], g) : -g;
        ce = -h * kLn2;
        const float back = exp2f(-d);
        ca = back * fmaf(-d, ce, ca);
        ce *= back;
        if (isnan(ll)) ca = ll;
        tg = (int)t;
      }
    }
    a.coefA[i] = ca;
    a.coefB[i] = cb;
    a.coefE[i] = ce;
    a.lseL[i] = ll;
    a.tgt[i] = tg;
    // |p log2 p| < 0.54
    dmax = fmaxf(dmax, fabsf(ca) + fabsf(cb) + 0.54f * fabsf(ce));
  }
  sm[tid] = dmax;
  sb[tid] = bad;
  __syncthreads();
  for (int w = 512; w > 0; w >>= 1) {
    if (tid < w) {
      sm[tid] = fmaxf(sm[tid], sm[tid + w]);
      sb[tid] |= sb[tid + w];
    }
    __syncthreads();
  }
  if (tid == 0) {
    a.status[0] = sb[0] ? FLCE_ERR_TARGET_OUT_OF_RANGE : FLCE_OK;
    int s = 0;
    const float bound = a.f16_d ? sm[0] * a.abs_scale : 0.0f;   // >= every |D|
    if (bound > 0.0f && isfinite(bound)) {
      int e;
      frexpf(bound, &e);
      s = min(max(14 - e, -120), 120);
    }
    a.dscale[0] = ldexpf(1.0f, s);
    a.dscale[1] = ldexpf(1.0f, -s);
  }
}

// The gradients, one vocabulary chunk after the other: the logit gradient, then the
// two contractions, each with large or small tiles as the plan says (D has one layout).
hipError_t launch_logprobs_backward(const Plan& pl, const LpPlan& lp, const LpGrad& g, const void* hidden,
                                    const void* weight, const void* bias, const void* targets, const float* lse,
                                    void* grad_hidden, void* grad_weight, void* grad_bias, char* ws, hipStream_t st) {
  LpPrepArgs a;
  a.targets = targets;
  a.tgt_i32 = pl.tgt_i32 ? 1 : 0;
  a.lse = lse;
  a.entropy = g.entropy;
  a.grad_logps = g.grad_logps;
  a.grad_entropy = g.grad_entropy;
  a.N = (int)pl.N;
  a.V = (int)pl.V;
  a.N_pad = (int)pl.N_pad;
  a.ignore_index = pl.ignore_index;
  a.coefA = reinterpret_cast<float*>(ws + pl.b_coefA);
  a.coefB = reinterpret_cast<float*>(ws + pl.b_coefB);
  a.coefE = reinterpret_cast<float*>(ws + lp.b_coefE);
  a.lseL = reinterpret_cast<float*>(ws + pl.b_lseL);
  a.tgt = reinterpret_cast<int*>(ws + pl.b_tgt);
  a.status = reinterpret_cast<int*>(ws);
  a.dscale = reinterpret_cast<float*>(ws + kDscaleOffset);
  a.f16_d = pl.dtype == FLCE_F16;
  a.abs_scale = fabsf(pl.scale);
  lp_prep_kernel<<<1, 1024, 0, st>>>(a);

  char* hiddenT = ws + pl.b_xt;
  if (pl.N > 0 && grad_weight) launch_transpose_hidden(pl.dtype, hidden, (int)pl.N, (int)pl.H, lp.K_pad, hiddenT, st, a.tgt, lp.split);
  float* gb_part = reinterpret_cast<float*>(ws + (lp.d_small ? lp.b_gbpart : pl.b_gbpart));
  const bool f32 = pl.dtype == FLCE_F32;
  for (int c = 0; c < pl.n_chunks; c++) {
    const int cv0 = (int)(c * pl.Vc);
    const int cvn = (int)(pl.V_pad - cv0 < pl.Vc ? pl.V_pad - cv0 : pl.Vc);
    if (pl.N > 0) {
      DlogitsArgs d;
      d.hidden = static_cast<const char*>(hidden);
      d.weight = static_cast<const char*>(weight);
      d.bias = bias;
      d.N = (int)pl.N;
      d.H = (int)pl.H;
      d.V = (int)pl.V;
      d.scale = pl.scale;
      d.cap = pl.cap;
      d.two_log2e_over_cap = pl.cap > 0 ? 2.0f * kLog2e / pl.cap : 0.0f;
      d.two_cap = 2.0f * pl.cap;
      d.cv0 = cv0;
      d.n_vt_c = lp.d_small ? cvn / 64 : cvn / 256;
      d.n_tt = lp.d_small ? lp.n64 : (int)pl.n_tt;
      d.coefA = a.coefA;
      d.coefB = a.coefB;
      d.coefE = a.coefE;
      d.lseL = a.lseL;
      d.tgt = a.tgt;
      d.D = ws + pl.b_D;
      d.ldD = (int)pl.Vc;
      d.gb_part = gb_part;
      d.ld_gb = (int)pl.V_pad;
      d.dscale = a.dscale;
      d.split = lp.split;
      if (lp.d_small) launch_dlogits_small(pl, d, st);
      else launch_lp_dlogits(pl, d, st);
    }
    GwArgs w;
    w.hiddenT = hiddenT;
    w.D = ws + pl.b_D;
    w.ldD = (int)pl.Vc;
    w.N = (int)pl.N;
    w.H = (int)pl.H;
    w.V = (int)pl.V;
    w.N_pad = lp.K_pad;
    w.cv0 = cv0;
    w.n_ht = lp.gw_small ? (int)((pl.H + 63) / 64) : (int)pl.n_ht;
    w.n_vt_c = lp.gw_small ? cvn / 64 : cvn / 256;
    w.gw = grad_weight;
    w.gw_type = pl.gw_dtype;
    w.dscale = a.dscale;
    w.accumulate = pl.accum_gw ? 1 : 0;
    w.acc32 = nullptr;
    w.mode = 3;
    if (grad_weight) {
      if (lp.gw_small) launch_gw_small(pl.dtype, w, st);
      else launch_gw(pl.dtype, w, st);
    }
    if (pl.N > 0 && grad_hidden) {
      GhArgs h;
      h.weight = static_cast<const char*>(weight);
      h.D = ws + pl.b_D;
      h.ldD = (int)pl.Vc;
      h.N = (int)pl.N;
      h.H = (int)pl.H;
      h.V = (int)pl.V;
      h.cv0 = cv0;
      h.cvn = cvn;
      h.n_ht = lp.gh_small ? (int)((pl.H + 63) / 64) : (int)pl.n_ht;
      h.n_tt = lp.split ? 2 * lp.n64 : (lp.gh_small ? lp.n64 : (int)pl.n_tt);
      h.split = lp.split;
      h.accb = f32 ? reinterpret_cast<float*>(grad_hidden) : reinterpret_cast<float*>(ws + pl.b_ghacc);
      h.out = grad_hidden;
      h.out_f32 = f32;
      h.mode = pl.n_chunks == 1 ? 3 : (c == 0 ? 0 : (c == pl.n_chunks - 1 ? 2 : 1));
      h.parts = lp.gh_small ? lp.gh_parts : pl.gh_parts;
      h.kt_per_part = lp.gh_small ? lp.gh_kt : pl.gh_kt_per_part;
      h.part = reinterpret_cast<float*>(ws + (lp.gh_small ? lp.b_ghpart : pl.b_ghpart));
      h.dscale = a.dscale;
      if (lp.gh_small) launch_gh_small(pl.dtype, h, st);
      else launch_gh(pl.dtype, h, st);
    }
  }
  if (grad_bias)
    launch_gb_reduce(pl.dtype, gb_part, lp.d_small ? lp.n64 : (int)pl.n_tt, (int)pl.V_pad, (int)pl.V, grad_bias,
                     pl.accum_gb ? 1 : 0, a.dscale, st);
  return hipGetLastError();
}

}  // namespace flce
