// The log-probability kernels with small tiles (flce_small.h), for problems whose
// 256 x 256 tiles would leave most CUs idle: few tokens, short vocabularies, and fp32,
// where one large tile takes a CU 0.2 ms per 1024 of hidden size.  The arithmetic of
// the epilogues is that of the large kernels (flce_logprobs.hip, flce_backward.hip).
#include "flce_logprobs.h"
#include "flce_lp_state.h"
#include "flce_small.h"

namespace flce {

using small::Shape;

// A workgroup's vocabulary tiles are one run of stages: the loads of the next tile's
// first stages are in flight during a tile's epilogue (4 tokens at H = 4096, V = 128256
// in 8 bits read 0.5 GB in 114 us with the merge, 4.6 TB/s; 136 us when the loads ran dry
// at every tile and workgroups came in more than one round).  Rows
// past V lie past the descriptor's end and read as 0.  Token tiles are the fast index:
// workgroups that share a weight tile run together.
template <typename T, bool HAS_BIAS, bool SOFTCAP, int BN>
__global__ __launch_bounds__(small::kThreadsS) void lp_small_kernel(LpTileArgs a, int n_tt) {
  typedef Shape<BN> Sh;
  constexpr int E = sizeof(T), MI = Sh::MI, NI = Sh::NI;
  constexpr int kStages = small::stages<T>(BN), SB = small::stage_bytes(BN);
  constexpr bool I8 = E == 1;
  typedef typename BiasOf<T>::type B;
  static __shared__ __attribute__((aligned(1024))) char lds[small::lds_bytes<T>(BN)];
  // a tile's bias and scales arrive with its first stage, up to kStages - 1 stages and so
  // as many tiles ahead of the tile in work
  static __shared__ __attribute__((aligned(256))) char bias_lds[kStages][256], scale_lds[kStages][256];
  float(&xs)[Sh::WM][4][BN] = *reinterpret_cast<float(*)[Sh::WM][4][BN]>(lds);   // after the last stage
  const int L = xcd_logical_id(blockIdx.x, gridDim.x);
  const int tt = L % n_tt, s = L / n_tt;
  const int vt_begin = (int)((int64_t)s * a.n_vt / a.S), vt_end = (int)((int64_t)(s + 1) * a.n_vt / a.S);
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  const int t0 = tt * BN;
  if (blockIdx.x == 0 && tid == 0) a.status[0] = FLCE_OK;

  const float s_u = SOFTCAP ? a.scale / a.cap : a.scale * kLog2e;   // as in lp_tiles_kernel
  const float cap2 = a.cap * kLog2e;
  LpState st[NI];
  int tgt[NI];
  float s_a[NI];
#pragma unroll
  for (int ni = 0; ni < NI; ni++) {
    st[ni] = LpState{kMasked, 0.0f, 0.0f, -INFINITY};
    const int t = t0 + (wn * NI + ni) * 16 + (lane & 15);
    const int64_t tv = t < a.N ? load_target(a.targets, t, a.tgt_i32) : a.ignore_index;
    tgt[ni] = (tv != a.ignore_index && tv >= 0 && tv < a.V) ? (int)tv : -1;
    s_a[ni] = I8 ? s_u * (t < a.N ? a.hidden_scale[t] : 0.0f) : s_u;
  }

  const uint32_t ld = (uint32_t)a.H * E;
  const int v_begin = a.v_first + vt_begin * 64, v_end = min(a.v_first + vt_end * 64, a.V);
  OperandDesc da, db;
  da.base = a.weight + (size_t)v_begin * ld;
  da.ld_bytes = ld;
  da.nrec = (uint32_t)(v_end - v_begin) * ld;
  da.cols_valid = 0;
  da.k_bytes = a.H * E;
  db.base = a.hidden + (size_t)t0 * ld;
  db.ld_bytes = ld;
  db.nrec = (uint32_t)min(a.N - t0, BN) * ld;
  db.cols_valid = 0;
  db.k_bytes = a.H * E;
  const int KT = (a.H * E + kBKB - 1) / kBKB, tiles = vt_end - vt_begin;
  small::Loader<T, true, small::kBMs> la;
  small::Loader<T, true, BN> lb;
  la.init(da, tid);
  lb.init(db, tid);
  const uint32_t lds0 = lds_addr_of(lds);

  int l_tile = 0, l_kt = 0, l_buf = 0, l_side = 0;   // the next stage to load
  auto load_next = [&]() {
    if (l_tile >= tiles) return;
    if (l_kt == 0) {   // (bytes past the last row's arrive as 0, whole words: see fwd_tiles_kernel)
      const int v = v_begin + l_tile * 64, rows = min(v_end - v, 64);
      if (HAS_BIAS && wave == 2)
        dma_vector(reinterpret_cast<const B*>(a.bias) + v, ((uint32_t)rows * sizeof(B) + 3u) & ~3u, bias_lds[l_side],
                   256, lane);
      if (I8 && wave == 3) dma_vector(a.weight_scale + v, (uint32_t)rows * 4, scale_lds[l_side], 256, lane);
    }
    const uint32_t to = lds0 + l_buf * SB;
    la.load(l_kt, to, (uint32_t)l_tile * 64u * ld);
    lb.load(l_kt, to + small::kStageA);
    l_buf = l_buf == kStages - 1 ? 0 : l_buf + 1;
    if (++l_kt == KT) {
      l_kt = 0;
      l_tile++;
      l_side = l_side == kStages - 1 ? 0 : l_side + 1;
    }
  };
#pragma unroll
  for (int p = 0; p < kStages - 1; p++) load_next();

  int buf = 0, left = tiles * KT;   // stages not yet consumed
  for (int tile = 0, side = 0; tile < tiles; tile++, side = side == kStages - 1 ? 0 : side + 1) {
    const int v0 = v_begin + tile * 64;
    Acc acc[MI][NI];
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
      for (int ni = 0; ni < NI; ni++) acc[mi][ni] = Acc{0.0f, 0.0f, 0.0f, 0.0f};
    small::in_blocks<T, BN>(KT, acc, [&](int kt, int end, Acc (&to)[MI][NI]) {
      for (; kt < end; kt++, left--) {
        if (left >= kStages - 1) small::wait_stage<T, true, true, BN, kStages - 2>(lb.loads);
        else wait_loads();
        __syncthreads();   // the stage has landed for every wave, and every wave has read the one before
        load_next();       // into the buffer of the one before
        small::stage_mma<T, true, true, BN>(lds + buf * SB, wm, wn, lane, to);
        buf = buf == kStages - 1 ? 0 : buf + 1;
      }
    });

    float sb[MI][4], ws[MI][4];
#pragma unroll
    for (int mi = 0; mi < MI; mi++) {
      const int row = (wm * MI + mi) * 16 + 4 * (lane >> 4);
      if constexpr (HAS_BIAS) {
        lds_vec4<B>(bias_lds[side], row, sb[mi]);
#pragma unroll
        for (int r = 0; r < 4; r++) sb[mi][r] *= s_u;
      }
      if constexpr (I8) lds_vec4<float>(scale_lds[side], row, ws[mi]);
    }
    float size = 0.0f;
#pragma unroll
    for (int ni = 0; ni < NI; ni++)
#pragma unroll
      for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          float u = I8 ? (float)__builtin_bit_cast(int, (float)acc[mi][ni][r]) * ws[mi][r] : acc[mi][ni][r];
          u = HAS_BIAS ? fmaf(u, s_a[ni], sb[mi][r]) : u * s_a[ni];
          acc[mi][ni][r] = u;
          size = fmaxf(size, fabsf(u));
        }
    const bool wide = SOFTCAP && __builtin_amdgcn_ballot_w64(size > kTanhNear) != 0;
#pragma unroll
    for (int ni = 0; ni < NI; ni++) {
      float mu = kMasked;
#pragma unroll
      for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          float u = acc[mi][ni][r];
          if constexpr (SOFTCAP) u = cap2 * (wide ? tanh_of<true>(u) : tanh_of<false>(u));
          const int v = v0 + (wm * MI + mi) * 16 + 4 * (lane >> 4) + r;
          if (v == tgt[ni]) st[ni].yt = u;
          if (v >= a.V) u = 2.0f * kMasked;   // below every running maximum: adds 0
          acc[mi][ni][r] = u;
          mu = fmaxf(mu, u);
        }
      const float m_new = fmaxf(st[ni].m, mu);
      const float dm = st[ni].l == 0.0f ? 0.0f : st[ni].m - m_new;
      const float alpha = fast_exp2(dm);
      float se = 0.0f, sx = 0.0f;
#pragma unroll
      for (int mi = 0; mi < MI; mi++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const float x = acc[mi][ni][r] - m_new, e = fast_exp2(x);
          se += e;
          sx = fmaf(e, fmaxf(x, kMasked), sx);
        }
      st[ni].T = fmaf(fmaf(dm, st[ni].l, st[ni].T), alpha, sx);
      st[ni].l = fmaf(st[ni].l, alpha, se);
      st[ni].m = m_new;
    }
  }

  __syncthreads();   // every wave has read the last stage
#pragma unroll
  for (int ni = 0; ni < NI; ni++) {
#pragma unroll
    for (int x = 16; x <= 32; x <<= 1) {
      LpState o;
      o.m = __shfl_xor(st[ni].m, x);
      o.l = __shfl_xor(st[ni].l, x);
      o.T = __shfl_xor(st[ni].T, x);
      o.yt = __shfl_xor(st[ni].yt, x);
      lp_merge(st[ni], o);
    }
    if (lane < 16) {
      const int c = (wn * NI + ni) * 16 + lane;
      xs[wm][0][c] = st[ni].m;
      xs[wm][1][c] = st[ni].l;
      xs[wm][2][c] = st[ni].T;
      xs[wm][3][c] = st[ni].yt;
    }
  }
  __syncthreads();
  if (tid < BN) {
    LpState r{xs[0][0][tid], xs[0][1][tid], xs[0][2][tid], xs[0][3][tid]};
#pragma unroll
    for (int w = 1; w < Sh::WM; w++) lp_merge(r, LpState{xs[w][0][tid], xs[w][1][tid], xs[w][2][tid], xs[w][3][tid]});
    const size_t plane = (size_t)a.S_all * a.N_pad;
    float* out = a.part + (size_t)(a.s_first + s) * a.N_pad + t0 + tid;
    out[0] = r.m;
    out[plane] = r.l;
    out[2 * plane] = r.T;
    out[3 * plane] = r.yt;
  }
}

// ---------------------------------------------------------------------------
// Logit gradient (with the entropy term): one 64 (vocabulary) x 64 (token) tile.
// ---------------------------------------------------------------------------
template <typename T> __device__ __forceinline__ void put4(T* p, const float* v) {
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 o;
#pragma unroll
  for (int j = 0; j < 4; j++) o[j] = (T)v[j];
  *reinterpret_cast<V4*>(p) = o;
}
template <typename T> __device__ __forceinline__ void get4(const T* p, float* v) {
  typedef T V4 __attribute__((ext_vector_type(4)));
  const V4 o = *reinterpret_cast<const V4*>(p);
#pragma unroll
  for (int j = 0; j < 4; j++) v[j] = (float)o[j];
}

template <typename T, bool HAS_BIAS, bool SOFTCAP>
__global__ __launch_bounds__(small::kThreadsS) void dlogits_small_kernel(DlogitsArgs a) {
  typedef Shape<64> Sh;
  constexpr int E = sizeof(T), MI = Sh::MI, NI = Sh::NI;
  static __shared__ __attribute__((aligned(1024))) char lds[small::lds_bytes<T>(64)];
  static __shared__ float gbs[Sh::WN][64];
  const int L = xcd_logical_id(blockIdx.x, gridDim.x);
  const int tt = L % a.n_tt, vt = L / a.n_tt;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  const int v0 = a.cv0 + vt * 64, t0 = tt * 64;
  const uint32_t ld = (uint32_t)a.H * E;
  OperandDesc da, db;
  da.base = a.weight + (size_t)v0 * ld;
  da.ld_bytes = ld;
  da.nrec = (uint32_t)max(min(a.V - v0, 64), 0) * ld;
  da.cols_valid = 0;
  da.k_bytes = a.H * E;
  db.base = a.hidden + (size_t)t0 * ld;
  db.ld_bytes = ld;
  db.nrec = (uint32_t)max(min(a.N - t0, 64), 0) * ld;
  db.cols_valid = 0;
  db.k_bytes = a.H * E;
  Acc acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; mi++)
#pragma unroll
    for (int ni = 0; ni < NI; ni++) acc[mi][ni] = Acc{0.0f, 0.0f, 0.0f, 0.0f};
  small::mainloop<T, true, true, 64>(da, db, (a.H * E + kBKB - 1) / kBKB, lds, acc);

  // with the cap u = v / cap, z = cap tanh(u) and softcap' = 1 - tanh^2(u)
  // without it u = y, as in the forward (bwd_dlogits_kernel has the reason)
  const float s2 = SOFTCAP ? a.scale / a.cap : a.scale * kLog2e;
  const float cap2 = a.cap * kLog2e;
  const float cmul = a.scale * a.dscale[0];
  float size = 0.0f;
#pragma unroll
  for (int ni = 0; ni < NI; ni++)
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        float u = acc[mi][ni][r] * s2;
        if (HAS_BIAS) {
          const int v = min(v0 + (wm * MI + mi) * 16 + 4 * (lane >> 4) + r, a.V - 1);
          u = fmaf(acc[mi][ni][r], s2, (float)reinterpret_cast<const T*>(a.bias)[v] * s2);
        }
        if (SOFTCAP) u = fmaxf(u, kMasked);   // (not NaN: see bwd_dlogits_kernel, ENTROPY)
        acc[mi][ni][r] = u;
        size = fmaxf(size, fabsf(u));
      }
  const bool wide = SOFTCAP && __builtin_amdgcn_ballot_w64(size > kTanhNear) != 0;
  T* D = reinterpret_cast<T*>(a.D);
  float cs[MI][4];
#pragma unroll
  for (int mi = 0; mi < MI; mi++)
#pragma unroll
    for (int r = 0; r < 4; r++) cs[mi][r] = 0.0f;
#pragma unroll
  for (int ni = 0; ni < NI; ni++) {
    const int t = t0 + (wn * NI + ni) * 16 + (lane & 15);   // the per-token arrays hold whole 256-token tiles
    const float cA = a.coefA[t] * cmul, cB = a.coefB[t] * cmul, cE = a.coefE[t] * cmul, lL = a.lseL[t];
    const int tg = a.tgt[t];
#pragma unroll
    for (int mi = 0; mi < MI; mi++) {
      const int vl = (wm * MI + mi) * 16 + 4 * (lane >> 4);
      float d[4];
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int v = v0 + vl + r;
        const float u = acc[mi][ni][r];
        if constexpr (SOFTCAP) {
          float f;
          const float x = fmaf(cap2, wide ? tanh_of<true>(u, &f) : tanh_of<false>(u, &f), -lL);
          d[r] = (fast_exp2(x) * fmaf(x, cE, cA)) * f;
          if (v == tg) d[r] -= cB * f;
        } else {
          const float x = fmaxf(u - lL, kMasked);
          d[r] = fast_exp2(x) * fmaf(x, cE, cA);
          if (v == tg) d[r] -= cB;
        }
        if (v >= a.V) d[r] = 0.0f;
        cs[mi][r] += d[r];
      }
      if (sizeof(T) == 2 && a.split) {
        // two rows: the rounded value and the rest
        T* row = D + (size_t)(2 * t) * a.ldD + (v0 - a.cv0) + vl;
        float rest[4];
#pragma unroll
        for (int r = 0; r < 4; r++) rest[r] = d[r] - (float)(T)d[r];
        put4<T>(row, d);
        put4<T>(row + a.ldD, rest);
      } else {
        put4<T>(D + (size_t)t * a.ldD + (v0 - a.cv0) + vl, d);
      }
    }
  }
  if constexpr (HAS_BIAS) {
    // column sums over the tile's 64 tokens: 16 lanes, then the two token waves
#pragma unroll
    for (int mi = 0; mi < MI; mi++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        float x = cs[mi][r];
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) x += __shfl_xor(x, o);
        if ((lane & 15) == 0) gbs[wn][(wm * MI + mi) * 16 + 4 * (lane >> 4) + r] = x;
      }
    __syncthreads();
    if (tid < 64) a.gb_part[(size_t)tt * a.ld_gb + v0 + tid] = gbs[0][tid] + gbs[1][tid];
  }
}

// ---------------------------------------------------------------------------
// grad_weight[v][h] = sum_t hidden[t][h] D[t][v]: a 64 (h) x 64 (v) tile.
// ---------------------------------------------------------------------------
template <typename T, typename OutT>
__global__ __launch_bounds__(small::kThreadsS) void gw_small_kernel(GwArgs a) {
  typedef Shape<64> Sh;
  constexpr int E = sizeof(T), MI = Sh::MI, NI = Sh::NI;
  static __shared__ __attribute__((aligned(1024))) char lds[small::lds_bytes<T>(64)];
  const int L = xcd_logical_id(blockIdx.x, gridDim.x);
  const int ht = L % a.n_ht, vt = L / a.n_ht;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  const int h0 = ht * 64, vl0 = vt * 64;
  OperandDesc da, db;
  const uint32_t ldt = (uint32_t)a.N_pad * E, ldd = (uint32_t)a.ldD * E;
  da.base = a.hiddenT + (size_t)h0 * ldt;
  da.ld_bytes = ldt;
  da.nrec = (uint32_t)min(a.H - h0, 64) * ldt;
  da.cols_valid = 0;
  da.k_bytes = a.N_pad * E;
  db.base = a.D + (size_t)vl0 * E;
  db.ld_bytes = ldd;
  db.nrec = a.N_pad > 0 ? (uint32_t)((size_t)a.N_pad * ldd - (size_t)vl0 * E) : 0u;
  db.cols_valid = a.ldD - vl0;
  db.k_bytes = 0;
  Acc acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; mi++)
#pragma unroll
    for (int ni = 0; ni < NI; ni++) acc[mi][ni] = Acc{0.0f, 0.0f, 0.0f, 0.0f};
  small::mainloop<T, true, false, 64>(da, db, (a.N_pad * E + kBKB - 1) / kBKB, lds, acc);
  const float inv = a.dscale[1];
  OutT* gw = reinterpret_cast<OutT*>(a.gw);
#pragma unroll
  for (int ni = 0; ni < NI; ni++) {
    const int v = a.cv0 + vl0 + (wn * NI + ni) * 16 + (lane & 15);
#pragma unroll
    for (int mi = 0; mi < MI; mi++) {
      const int h = h0 + (wm * MI + mi) * 16 + 4 * (lane >> 4);   // 4 consecutive h; H % 8 == 0
      if (v >= a.V || h >= a.H) continue;
      float c[4], prev[4];
#pragma unroll
      for (int r = 0; r < 4; r++) c[r] = acc[mi][ni][r] * inv;
      if (a.accumulate) {
        get4<OutT>(gw + (size_t)v * a.H + h, prev);
#pragma unroll
        for (int r = 0; r < 4; r++) c[r] += prev[r];
      }
      put4<OutT>(gw + (size_t)v * a.H + h, c);
    }
  }
}

// ---------------------------------------------------------------------------
// grad_hidden[t][h] = sum_v weight[v][h] D[t][v] over a chunk: a 64 (h) x 64 (t) tile
// of one split of the vocabulary; modes and parts as bwd_gh_kernel.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(small::kThreadsS) void gh_small_kernel(GhArgs a) {
  typedef Shape<64> Sh;
  constexpr int E = sizeof(T), MI = Sh::MI, NI = Sh::NI;
  static __shared__ __attribute__((aligned(1024))) char lds[small::lds_bytes<T>(64)];
  const int L = xcd_logical_id(blockIdx.x, gridDim.x);
  const int n_tiles = a.n_ht * a.n_tt, split = L / n_tiles, in = L - split * n_tiles;
  const int tt = in % a.n_tt, ht = in / a.n_tt;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  const int h0 = ht * 64, t0 = tt * 64;
  const int KT_all = (a.cvn * E + kBKB - 1) / kBKB;
  const int kt0 = split * a.kt_per_part;
  const int KT = max(min(KT_all - kt0, a.kt_per_part), 0);
  const int v_off = kt0 * (kBKB / E);
  OperandDesc da, db;
  const uint32_t ldw = (uint32_t)a.H * E, ldd = (uint32_t)a.ldD * E;
  const int vrows = max(min(a.V - a.cv0, a.cvn) - v_off, 0);
  da.base = a.weight + ((size_t)(a.cv0 + v_off) * a.H + h0) * E;
  da.ld_bytes = ldw;
  da.nrec = vrows > 0 ? (uint32_t)((size_t)vrows * ldw - (size_t)h0 * E) : 0u;
  da.cols_valid = a.H - h0;
  da.k_bytes = 0;
  db.base = a.D + (size_t)t0 * ldd + (size_t)v_off * E;
  db.ld_bytes = ldd;
  db.nrec = 64u * ldd - (uint32_t)v_off * E;
  db.cols_valid = 0;
  db.k_bytes = (a.cvn - v_off) * E;
  Acc acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; mi++)
#pragma unroll
    for (int ni = 0; ni < NI; ni++) acc[mi][ni] = Acc{0.0f, 0.0f, 0.0f, 0.0f};
  small::mainloop<T, false, true, 64>(da, db, KT, lds, acc);
  const float inv = a.dscale[1];
#pragma unroll
  for (int ni = 0; ni < NI; ni++) {
    const int row = t0 + (wn * NI + ni) * 16 + (lane & 15), t = a.split ? row >> 1 : row;
#pragma unroll
    for (int mi = 0; mi < MI; mi++) {
      float c[4], prev[4];
#pragma unroll
      for (int r = 0; r < 4; r++) c[r] = acc[mi][ni][r] * inv;
      if (a.split) {   // a token's two rows are neighbouring columns here
#pragma unroll
        for (int r = 0; r < 4; r++) c[r] += __shfl_xor(c[r], 1);
      }
      const int h = h0 + (wm * MI + mi) * 16 + 4 * (lane >> 4);
      if (t >= a.N || h >= a.H || (a.split && (row & 1))) continue;
      const size_t o = (size_t)t * a.H + h;
      if (a.parts > 1) {   // partial of this split; the reduction applies the mode
        put4<float>(a.part + (size_t)split * a.N * a.H + o, c);
        continue;
      }
      if (a.mode == 1 || a.mode == 2) {
        get4<float>(a.accb + o, prev);
#pragma unroll
        for (int r = 0; r < 4; r++) c[r] += prev[r];
      }
      if (a.mode <= 1 || a.out_f32) put4<float>((a.mode <= 1 ? a.accb : reinterpret_cast<float*>(a.out)) + o, c);
      else put4<T>(reinterpret_cast<T*>(a.out) + o, c);
    }
  }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------
template <typename T, int BN> static void lp_small_t(const Plan& pl, const LpTileArgs& a, int n_tt, hipStream_t st) {
  const int nwg = n_tt * a.S;
  if (pl.has_bias) {
    if (pl.cap > 0) lp_small_kernel<T, true, true, BN><<<nwg, small::kThreadsS, 0, st>>>(a, n_tt);
    else lp_small_kernel<T, true, false, BN><<<nwg, small::kThreadsS, 0, st>>>(a, n_tt);
  } else {
    if (pl.cap > 0) lp_small_kernel<T, false, true, BN><<<nwg, small::kThreadsS, 0, st>>>(a, n_tt);
    else lp_small_kernel<T, false, false, BN><<<nwg, small::kThreadsS, 0, st>>>(a, n_tt);
  }
}
template <typename T> static void lp_small_bn(const Plan& pl, int bn, const LpTileArgs& a, int n_tt, hipStream_t st) {
  if (bn == 16) lp_small_t<T, 16>(pl, a, n_tt, st);
  else lp_small_t<T, 64>(pl, a, n_tt, st);
}
void launch_lp_small(const Plan& pl, int bn, const LpTileArgs& a, int n_tt, hipStream_t st) {
  if (pl.int8) lp_small_bn<int8_t>(pl, bn, a, n_tt, st);
  else if (pl.dtype == FLCE_BF16) lp_small_bn<bf16>(pl, bn, a, n_tt, st);
  else if (pl.dtype == FLCE_F16) lp_small_bn<f16>(pl, bn, a, n_tt, st);
  else lp_small_bn<float>(pl, bn, a, n_tt, st);
}

template <typename T> static void dlogits_small_t(const Plan& pl, const DlogitsArgs& d, hipStream_t st) {
  const int nwg = d.n_vt_c * d.n_tt;
  if (pl.has_bias) {
    if (pl.cap > 0) dlogits_small_kernel<T, true, true><<<nwg, small::kThreadsS, 0, st>>>(d);
    else dlogits_small_kernel<T, true, false><<<nwg, small::kThreadsS, 0, st>>>(d);
  } else {
    if (pl.cap > 0) dlogits_small_kernel<T, false, true><<<nwg, small::kThreadsS, 0, st>>>(d);
    else dlogits_small_kernel<T, false, false><<<nwg, small::kThreadsS, 0, st>>>(d);
  }
}
void launch_dlogits_small(const Plan& pl, const DlogitsArgs& d, hipStream_t st) {
  if (pl.dtype == FLCE_BF16) dlogits_small_t<bf16>(pl, d, st);
  else if (pl.dtype == FLCE_F16) dlogits_small_t<f16>(pl, d, st);
  else dlogits_small_t<float>(pl, d, st);
}

template <typename T> static void gw_small_t(const GwArgs& g, hipStream_t st) {
  const int nwg = g.n_ht * g.n_vt_c;
  if (g.gw_type == FLCE_BF16) gw_small_kernel<T, bf16><<<nwg, small::kThreadsS, 0, st>>>(g);
  else if (g.gw_type == FLCE_F16) gw_small_kernel<T, f16><<<nwg, small::kThreadsS, 0, st>>>(g);
  else gw_small_kernel<T, float><<<nwg, small::kThreadsS, 0, st>>>(g);
}
void launch_gw_small(int dtype, const GwArgs& g, hipStream_t st) {
  if (dtype == FLCE_BF16) gw_small_t<bf16>(g, st);
  else if (dtype == FLCE_F16) gw_small_t<f16>(g, st);
  else gw_small_t<float>(g, st);
}

void launch_gh_small(int dtype, const GhArgs& h, hipStream_t st) {
  const int nwg = h.n_ht * h.n_tt * h.parts;
  if (dtype == FLCE_BF16) gh_small_kernel<bf16><<<nwg, small::kThreadsS, 0, st>>>(h);
  else if (dtype == FLCE_F16) gh_small_kernel<f16><<<nwg, small::kThreadsS, 0, st>>>(h);
  else gh_small_kernel<float><<<nwg, small::kThreadsS, 0, st>>>(h);
  if (h.parts > 1) launch_gh_reduce(dtype, h, st);
}

}  // namespace flce
