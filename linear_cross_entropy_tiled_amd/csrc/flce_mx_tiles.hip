// Log-probabilities from MXFP4 operands with 256 x 256 tiles: the counterpart of
// lp_tiles_kernel (flce_logprobs.hip has the epilogue's mathematics).
//
// The stages are those of the other types' loop (flce_device.h): 128 bytes of K a row, two
// buffers, loads a whole iteration ahead.  What differs:
//  - v_mfma_scale_f32_32x32x64_f8f6f4.  An instruction that carries scales takes twice the
//    issue slots of one without; the 32 x 32 form does the work of two 16 x 16 ones, and its
//    fragments are 24 registers a sub-step instead of 36.
//  - The scales come through LDS in the order of launch_mx_prep, 24 bytes a lane and
//    stage.
//  - A workgroup's vocabulary tiles are one run of stages: 16 stages at H = 4096 are so
//    short that the loads of a tile's first two, if nothing else ran, would be a tenth of it.
//  - The epilogue is a larger share (5 us of a tile's 34 at H = 4096, 10 of 28 at H = 2048
//    with bias and softcap, before it was cut): the sums begin with the bias, two logits share
//    a comparison, rows past V are masked in the last tile only.
//
// What bounds it: N = 8192, H = 4096, V = 128256 takes 1.89 to 2.1 ms, 4.1 to 4.6 PFLOP/s (the
// library's largest MXFP4 product 3.0), matrix units busy 65%, and the board's power: with 64
// stages of random data the clock is 1.56 GHz, of zeros 2.08 at the same cycles.  With few
// stages the epilogue: N = 1000, H = 2048, V = 50001, bias, softcap 68 us, units busy 33%.
// The steps there, whole calls in us: 64 x 64 tiles alone 6273 and 177; 256 x 256 with 16 x 16
// instructions 2204 and 103; 32 x 32 and one run of stages 2190 and 102, prepared in one launch
// 2140 and 100; the epilogue 2000 and 88.
#include <math.h>

#include <utility>

#include "flce_device.h"
#include "flce_logprobs.h"
#include "flce_lp_state.h"
#include "flce_mx_device.h"

namespace flce {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kMxM = 4, kMxN = 2;    // 32 x 32 tiles of a wave's 128 x 64
constexpr int kMxSub = 4;            // sub-steps of a stage, 64 values each

// f(integral constants 0 .. N - 1), in order.
template <typename F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F&& f) {
  each_of(std::make_integer_sequence<int, N>{}, f);
}

template <int SEL_A, int SEL_B>
__device__ __forceinline__ void mma_mx32(f32x16& c, const i32x4& a, const i32x4& b, int sa, int sb) {
  const i32x8 wide_a = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 wide_b = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide_a, wide_b, c, 4, 4, SEL_A, sa, SEL_B, sb);
}

// Rows r0 + lane % 32 of a stage's operand, chunk 2 s + lane / 32.
__device__ __forceinline__ i32x4 mx_fragment(const char* op, int r0, int s, int lane) {
  const int row = r0 + (lane & 31), kc = 2 * s + (lane >> 5);
  return *reinterpret_cast<const i32x4*>(op + row * kBKB + ((kc ^ ((row >> 1) & 7)) << 4));
}

struct MxFrags {
  i32x4 a[2][kMxM], b[2][kMxN];
};

// The matrix instructions of sub-step S with the fragments of buffer S % 2, while those of sub-step (S + 1) % 4 of
// `stage` are read into the other: B's with the first row of tiles, A's with the ones that follow.
template <int S>
__device__ __forceinline__ void mx_substep(MxFrags& f, const i32x4& sa, const i32x2& sb, const char* stage, int wm, int wn,
                                           int lane, f32x16 (&acc)[kMxM][kMxN]) {
  constexpr int kCur = S & 1, kNext = 1 - kCur, kS = (S + 1) % kMxSub;
  each<kMxM>([&](auto mi_) __attribute__((always_inline)) {
    constexpr int mi = decltype(mi_)::value;
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (mi == 0) {
#pragma unroll
      for (int ni = 0; ni < kMxN; ni++)
        f.b[kNext][ni] = mx_fragment(stage + kOperandStage, wn * kWaveN + 32 * ni, kS, lane);
    } else {
      f.a[kNext][mi - 1] = mx_fragment(stage, wm * kWaveM + 32 * (mi - 1), kS, lane);
      if constexpr (mi == kMxM - 1) f.a[kNext][mi] = mx_fragment(stage, wm * kWaveM + 32 * mi, kS, lane);
    }
    each<kMxN>([&](auto nj_) __attribute__((always_inline)) {
      constexpr int nj = decltype(nj_)::value, ni = (mi & 1) ? kMxN - 1 - nj : nj;
      mma_mx32<mi, 2 * (S & 1) + ni>(acc[mi][ni], f.a[kCur][mi], f.b[kCur][ni], sa[S], sb[S >> 1]);
    });
  });
  __builtin_amdgcn_sched_barrier(0);
}

// prefetch_stage of flce_device.h with one loader for both operands.
__device__ __forceinline__ bool mx_prefetch(const OperandLoader<mx4, true>& lo, const i32x4& rs_a, const i32x4& rs_b,
                                            const L2Share& sh, int kt, int wave, int lane) {
  if (wave >= kLoadWaves) return false;
  const bool is_a = wave < kLoadWaves / 2;
  const int n = is_a ? sh.a_n : sh.b_n, rank = is_a ? sh.a_rank : sh.b_rank;
  if (n < 2) return false;
  const int first = rank * 256 / n, count = (rank + 1) * 256 / n - first, off = (wave % (kLoadWaves / 2)) * 64;
  if (off >= count) return false;
  OperandLoader<mx4, true> p = lo;
  p.rsrc = is_a ? rs_a : rs_b;
  p.prefetch_line(kt, first + off + lane, off + lane < count,
                  __builtin_amdgcn_readfirstlane(lds_addr_of(g_prefetch_sink)));
  return true;
}

template <bool HAS_BIAS, bool SOFTCAP> __global__ __launch_bounds__(kThreads, 1) void mx_tiles_kernel(LpTileArgs a) {
  const int L = xcd_logical_id(blockIdx.x, gridDim.x);
  // the tile order of lp_tiles_kernel
  const int n_tt = (int)gridDim.x / a.S;
  const bool grouped = a.S % 8 == 0 && n_tt % 4 == 0 && gridDim.x >= 256;
  int tt, s;
  if (grouped) {
    grouped_tile(L, n_tt, a.S, 4, tt, s);
  } else {
    tt = L / a.S;
    s = L % a.S;
  }
  const int vt_begin = (int)((int64_t)s * a.n_vt / a.S), vt_end = (int)((int64_t)(s + 1) * a.n_vt / a.S);
  int tid = threadIdx.x;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const int t0 = tt * 256;
  if (blockIdx.x == 0 && tid == 0) a.status[0] = FLCE_OK;

  static __shared__ __attribute__((aligned(1024))) char scales[2][2 * kMxStage];
  static __shared__ __attribute__((aligned(16))) char bias_lds[2][HAS_BIAS ? 1024 : 16];

  LpState st[kMxN];
  int tgt[kMxN];
#pragma unroll
  for (int ni = 0; ni < kMxN; ni++) {
    st[ni] = LpState{kMasked, 0.0f, 0.0f, -INFINITY};
    const int t = t0 + wn * kWaveN + 32 * ni + (lane & 31);
    const int64_t tv = t < a.N ? load_target(a.targets, t, a.tgt_i32) : a.ignore_index;
    tgt[ni] = (tv != a.ignore_index && tv >= 0 && tv < a.V) ? (int)tv : -1;
  }

  const uint32_t ld = (uint32_t)a.H;
  const int KT = (a.H + kBKB - 1) / kBKB;
  // one loader for both operands, whose rows are equally long: only their descriptors differ
  OperandDesc d;
  d.base = a.hidden + (size_t)t0 * ld;
  d.ld_bytes = ld;
  d.nrec = (uint32_t)min(a.N - t0, 256) * ld;
  d.cols_valid = 0;
  d.k_bytes = a.H;
  OperandLoader<mx4, true> lo;
  lo.init(d, tid);
  const i32x4 rs_b = lo.rsrc;
  i32x4 rs_a = rs_b;
  const i32x4 rs_h = make_rsrc_words(a.hidden_tmx + (size_t)tt * KT * kMxStage, (uint32_t)KT * kMxStage);
  i32x4 rs_w = rs_h;
  const uint32_t mx_to = __builtin_amdgcn_readfirstlane(lds_addr_of(scales[0]) + wave * 1024);

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

  // the next stage to load: its tile's rows of the weight and their scales
  int l_vt = vt_begin, l_kt = 0, l_buf = 0;
  auto load_next = [&]() __attribute__((always_inline)) {
    if (l_vt == vt_end) return;
    if (l_kt == 0) {
      const int v0 = a.v_first + l_vt * 256;
      rs_a = make_rsrc_words(a.weight + (size_t)v0 * ld, (uint32_t)min(a.V - v0, 256) * ld);
      rs_w = make_rsrc_words(a.weight_tmx + (size_t)(v0 / 256) * KT * kMxStage, (uint32_t)KT * kMxStage);
      if (HAS_BIAS && wave == kLoadWaves)
        dma_vector(reinterpret_cast<const float*>(a.bias) + v0, (uint32_t)min(a.V - v0, 256) * 4,
                   bias_lds[(l_vt - vt_begin) & 1], 1024, lane);
    }
    if (wave < kLoadWaves) {
      char* stage = g_lds + l_buf * kStageBytes;
      lo.rsrc = rs_a;
      lo.load(l_kt, stage);
      lo.rsrc = rs_b;
      lo.load(l_kt, stage + kOperandStage);
      // 1 KiB of the scales each: the weight's two, the hidden states' two
      dma16(wave < 2 ? rs_w : rs_h, __builtin_amdgcn_readfirstlane(mx_to + l_buf * 2 * kMxStage), (uint32_t)(16 * lane),
            __builtin_amdgcn_readfirstlane((uint32_t)l_kt * kMxStage + (uint32_t)(wave & 1) * 1024));
    }
    l_buf ^= 1;
    if (++l_kt == KT) {
      l_kt = 0;
      l_vt++;
    }
  };

  // the accumulator times s_u is u = y, or with the cap u = v / cap, y = cap log2(e) tanh(u)
  const float s_u = SOFTCAP ? a.scale / a.cap : a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e;

  const char* sc_a = scales[0] + wm * 1024 + lane * 16;
  const char* sc_b = scales[0] + kMxStage + wn * 512 + lane * 8;
  load_next();
  wait_loads();
  __syncthreads();
  load_next();
  int buf = 0;
  bool pf = false;   // this wave's most recent vector-memory instruction is an L2 prefetch
  for (int vt = vt_begin; vt < vt_end; ++vt) {
    const int v0 = a.v_first + vt * 256;
    f32x16 acc[kMxM][kMxN];
    // the sums begin with the bias (a lane holds rows 32 mi + 8 q + 4 (lane / 32) + r in acc[mi][ni][4 q + r])
    const int lane_row = 4 * (lane >> 5);
#pragma unroll
    for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        float b4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (HAS_BIAS)
          lds_vec4<float>(bias_lds[(vt - vt_begin) & 1], wm * kWaveM + 32 * mi + 8 * q + lane_row, b4);
#pragma unroll
        for (int ni = 0; ni < kMxN; ni++)
#pragma unroll
          for (int r = 0; r < 4; r++) acc[mi][ni][4 * q + r] = b4[r];
      }
    // (the first fragments are read here, and not with the tile before's last ones, so that none is live in its
    // epilogue)
    MxFrags f;
    const char* first = g_lds + buf * kStageBytes;
#pragma unroll
    for (int ni = 0; ni < kMxN; ni++) f.b[0][ni] = mx_fragment(first + kOperandStage, wn * kWaveN + 32 * ni, 0, lane);
#pragma unroll
    for (int mi = 0; mi < kMxM; mi++) f.a[0][mi] = mx_fragment(first, wm * kWaveM + 32 * mi, 0, lane);
    i32x4 sa = *reinterpret_cast<const i32x4*>(sc_a + buf * 2 * kMxStage);
    i32x2 sb = *reinterpret_cast<const i32x2*>(sc_b + buf * 2 * kMxStage);
    for (int kt = 0; kt < KT; ++kt, buf ^= 1) {
      const char* cur = g_lds + buf * kStageBytes;
      const char* nxt = g_lds + (buf ^ 1) * kStageBytes;
      mx_substep<0>(f, sa, sb, cur, wm, wn, lane, acc);
      mx_substep<1>(f, sa, sb, cur, wm, wn, lane, acc);
      mx_substep<2>(f, sa, sb, cur, wm, wn, lane, acc);
      // (else the compiler moves these sub-steps' matrix instructions past the branches below, away from the reads that
      // they are to cover)
#pragma unroll
      for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
        for (int ni = 0; ni < kMxN; ni++) asm volatile("" : "+v"(acc[mi][ni]));
      // the next stage must be in LDS; a prefetch issued after it may still be in flight
      if (pf) wait_vmcnt_1();
      else wait_loads();
      __syncthreads();
      load_next();   // into this stage's buffer, whose last fragments are in registers
      pf = kt + kPrefetchAhead < KT &&
           mx_prefetch(lo, rs_a, rs_b, sh, kt + kPrefetchAhead, wave, lane);
      // (after the last stage of all these reads find stale LDS, which is not used)
      const i32x4 sa_next = *reinterpret_cast<const i32x4*>(sc_a + (buf ^ 1) * 2 * kMxStage);
      const i32x2 sb_next = *reinterpret_cast<const i32x2*>(sc_b + (buf ^ 1) * 2 * kMxStage);
      mx_substep<3>(f, sa, sb, nxt, wm, wn, lane, acc);
      sa = sa_next;
      sb = sb_next;
    }

    // A lane holds 64 rows of each of its two token columns.  y replaces the sums.
    const int vw = v0 + wm * kWaveM;
    const int n_valid = a.V - vw;
#pragma unroll
    for (int ni = 0; ni < kMxN; ni++) {
#pragma unroll
      for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          float u[4];
#pragma unroll
          for (int r = 0; r < 4; r++) u[r] = acc[mi][ni][4 * q + r] * s_u;
          if constexpr (SOFTCAP) {
            float th[4];
            tanh4(u, th);
#pragma unroll
            for (int r = 0; r < 4; r++) u[r] = cap2 * th[r];
          }
#pragma unroll
          for (int r = 0; r < 4; r++) acc[mi][ni][4 * q + r] = u[r];
        }
      if (n_valid < kWaveM) {
        // rows past V lie below every maximum and add 0.  (Their number is opaque, or the comparisons of both columns
        // are made together and 128 scalar registers kept for them.)
        int lim = n_valid - lane_row;
        asm volatile("" : "+v"(lim));
#pragma unroll
        for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
          for (int i = 0; i < 16; i++)
            if (32 * mi + 8 * (i >> 2) + (i & 3) >= lim) acc[mi][ni][i] = 2.0f * kMasked;
      }
      float mu = kMasked;   // stays where there is no finite logit
#pragma unroll
      for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
        for (int i = 0; i < 16; i++) mu = fmaxf(mu, acc[mi][ni][i]);
      const int rel = tgt[ni] - vw;
      const bool hit = rel >= 0 && rel < kWaveM && ((rel >> 2) & 1) == (lane >> 5);
      if (__builtin_amdgcn_ballot_w64(hit)) {
        int rel_l = rel - lane_row;
        asm volatile("" : "+v"(rel_l));
        float yt = 0.0f;
#pragma unroll
        for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
          for (int i = 0; i < 16; i++)
            if (32 * mi + 8 * (i >> 2) + (i & 3) == rel_l) yt = acc[mi][ni][i];
        if (hit) st[ni].yt = yt;
      }
      const float m_new = fmaxf(st[ni].m, mu);
      const float dm = st[ni].l == 0.0f ? 0.0f : st[ni].m - m_new;
      const float alpha = fast_exp2(dm);
      float se0 = 0.f, se1 = 0.f, sx0 = 0.f, sx1 = 0.f;
#pragma unroll
      for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const float x = acc[mi][ni][i] - m_new, e = fast_exp2(x);
          if (i & 1) {
            se1 += e;
            sx1 = fmaf(e, x, sx1);
          } else {
            se0 += e;
            sx0 = fmaf(e, x, sx0);
          }
        }
      float sx = sx0 + sx1;
      // a logit of -inf (a bias, or a sum past fp32's range) is to add 0 and not 0 times infinity: seldom, so the sum is
      // formed again.  (A maximum per logit takes 1 to 4%, this half of it; both columns' sums in one place spill.)
      if (!SOFTCAP && __builtin_amdgcn_ballot_w64(sx != sx)) {
        float again = 0.0f;
#pragma unroll
        for (int mi = 0; mi < kMxM; mi++)
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const float x = acc[mi][ni][i] - m_new;
            again = fmaf(fast_exp2(x), fmaxf(x, kMasked), again);
          }
        sx = sx != sx ? again : sx;   // (a column's sum does not depend on its neighbours)
      }
      st[ni].T = fmaf(fmaf(dm, st[ni].l, st[ni].T), alpha, sx);
      st[ni].l = fmaf(st[ni].l, alpha, se0 + se1);
      st[ni].m = m_new;
    }
  }

  // the two lanes of a token column, then the two M waves, through LDS
  __syncthreads();   // every wave has made its last read of the stages
  float* xs = reinterpret_cast<float*>(g_stage0);   // [wn][field][kWaveN]
#pragma unroll
  for (int ni = 0; ni < kMxN; ni++) {
    LpState o;
    o.m = __shfl_xor(st[ni].m, 32);
    o.l = __shfl_xor(st[ni].l, 32);
    o.T = __shfl_xor(st[ni].T, 32);
    o.yt = __shfl_xor(st[ni].yt, 32);
    lp_merge(st[ni], o);
    if (wm == 1 && lane < 32) {
      float* p = xs + wn * 4 * kWaveN + 32 * ni + lane;
      p[0 * kWaveN] = st[ni].m;
      p[1 * kWaveN] = st[ni].l;
      p[2 * kWaveN] = st[ni].T;
      p[3 * kWaveN] = st[ni].yt;
    }
  }
  __syncthreads();
  if (wm == 0 && lane < 32) {
    const size_t plane = (size_t)a.S_all * a.N_pad;
#pragma unroll
    for (int ni = 0; ni < kMxN; ni++) {
      const int c = 32 * ni + lane;
      const float* p = xs + wn * 4 * kWaveN + c;
      lp_merge(st[ni], LpState{p[0 * kWaveN], p[1 * kWaveN], p[2 * kWaveN], p[3 * kWaveN]});
      float* out = a.part + (size_t)(a.s_first + s) * a.N_pad + t0 + wn * kWaveN + c;
      out[0] = st[ni].m;
      out[plane] = st[ni].l;
      out[2 * plane] = st[ni].T;
      out[3 * plane] = st[ni].yt;
    }
  }
}

void launch_mx_tiles(const Plan& pl, const LpTileArgs& a, int nwg, hipStream_t st) {
  if (pl.has_bias) {
    if (pl.cap > 0) mx_tiles_kernel<true, true><<<nwg, kThreads, 0, st>>>(a);
    else mx_tiles_kernel<true, false><<<nwg, kThreads, 0, st>>>(a);
  } else {
    if (pl.cap > 0) mx_tiles_kernel<false, true><<<nwg, kThreads, 0, st>>>(a);
    else mx_tiles_kernel<false, false><<<nwg, kThreads, 0, st>>>(a);
  }
}

}  // namespace flce
