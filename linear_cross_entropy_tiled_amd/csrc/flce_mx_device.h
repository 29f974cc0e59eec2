// MXFP4 operands in the matrix loops (flce_mx.h has the format).
#pragma once

#include <utility>

#include "flce_device.h"
#include "flce_mx.h"

namespace flce {

template <> struct Frag<mx4, true> : Frag16K<i32x4> {};

// c += a b over 128 of K; a lane's fragment is one block, whose scale is byte SEL of sa (sb).
template <int SEL_A, int SEL_B>
__device__ __forceinline__ void mma_mx(Acc& c, const i32x4& a, const i32x4& b, int sa, int sb) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));   // the 4-bit types use the low four registers
  const i32x8 wide_a = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 wide_b = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide_a, wide_b, c, 4, 4, SEL_A, sa, SEL_B, sb);
}

// 4-byte direct-to-LDS load (dma16 has the rules): lane l's word lands at lds_addr + 4 l.
__device__ __forceinline__ void dma4(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory");
}

// f(integral constants 0 .. N - 1), in order.
template <typename F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F&& f) {
  each_of(std::make_integer_sequence<int, N>{}, f);
}

// ---------------------------------------------------------------------------
// The 256 x 256 loop (tile_mainloop of flce_device.h) of MXFP4 operands.  The stages,
// fragments and their order in time are the same.  The scales come from a copy of them in
// the order in which the matrix instructions want them (mx_tile_kernel): of a tile's stage,
// for each sub-step, each 64 rows and each lane one word, whose byte j is the scale of row
// 16 j + lane % 16, block 4 s + lane / 16.  So a wave reads three words a lane and sub-step
// (two for its 128 rows of A, one for its 64 of B) for 32 matrix instructions, which pick
// their byte; one byte a fragment out of rows as they are stored would be 12 reads.
// ---------------------------------------------------------------------------
constexpr int kMxStage = 2048;   // a tile's scales of a stage: 2 sub-steps x 4 x 64 words
static __shared__ __attribute__((aligned(1024))) char g_mx_lds[2 * 2 * kMxStage];

struct MxFrags {
  i32x4 a[kMI + 1];
  i32x4 b[2][kNI];
  int sa[2][2], sb[2];   // by sub-step

  __device__ __forceinline__ void read_a(const char* stage, int s, int mi, int slot, int wm, int lane) {
    a[slot] = Frag<mx4, true>::read(stage, wm * kWaveM + mi * 16, s, lane);
  }
  template <int BUF>
  __device__ __forceinline__ void read_b(const char* stage, const char* sc, int s, int wm, int wn, int lane) {
    const int* w = reinterpret_cast<const int*>(sc) + s * 256 + lane;
    sa[BUF][0] = w[128 * wm];
    sa[BUF][1] = w[128 * wm + 64];
    sb[BUF] = w[kMxStage / 4 + 64 * wn];
#pragma unroll
    for (int i = 0; i < kNI; i++)
      b[BUF][i] = Frag<mx4, true>::read(stage + kOperandStage, wn * kWaveN + i * 16, s, lane);
  }
};

// substep of flce_device.h.
template <int CUR>
__device__ __forceinline__ void substep_mx(MxFrags& f, const char* stage, const char* sc, int s, int wm, int wn, int lane,
                                           Acc (&acc)[kMI][kNI]) {
  constexpr int kLastCur = kMI - 1 + CUR, kLastNext = kMI - CUR;
  __builtin_amdgcn_sched_barrier(0);
  f.template read_b<1 - CUR>(stage, sc, s, wm, wn, lane);
  each<kMI>([&](auto mi_) __attribute__((always_inline)) {
    constexpr int mi = decltype(mi_)::value, slot = mi == kMI - 1 ? kLastCur : mi;
    if constexpr (mi > 0) {
      f.read_a(stage, s, mi - 1, mi - 1, wm, lane);
      if constexpr (mi == kMI / 2) f.read_a(stage, s, kMI - 1, kLastNext, wm, lane);
    }
    each<kNI>([&](auto nj_) __attribute__((always_inline)) {
      constexpr int nj = decltype(nj_)::value, ni = (mi & 1) ? kNI - 1 - nj : nj;
      mma_mx<(mi & 3), ni>(acc[mi][ni], f.a[slot], f.b[CUR][ni], f.sa[CUR][mi >> 2], f.sb[CUR]);
    });
    __builtin_amdgcn_sched_barrier(0);
  });
}

// mx_a, mx_b: the tiles' scales, kMxStage bytes a stage.
__device__ __forceinline__ void tile_mainloop_mx(const OperandDesc& da, const OperandDesc& db, const uint8_t* mx_a,
                                                 const uint8_t* mx_b, int KT, const L2Share& sh, Acc (&acc)[kMI][kNI]) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int wm = wave / kWavesN, wn = wave % kWavesN;

  OperandLoader<mx4, true> la, lb;
  la.init(da, tid);
  lb.init(db, tid);
  // one piece of 1 KiB for each loading wave: A's two, B's two
  const i32x4 rs = make_rsrc_words(la.wave < 2 ? mx_a : mx_b, (uint32_t)KT * kMxStage);
  const uint32_t mx_to = __builtin_amdgcn_readfirstlane(lds_addr_of(g_mx_lds) + la.wave * 1024);
  const uint32_t mx_off = (uint32_t)(16 * lane);
  auto load = [&](int kt, int buf) __attribute__((always_inline)) {
    char* stage = g_lds + buf * kStageBytes;
    la.load(kt, stage);
    lb.load(kt, stage + kOperandStage);
    if (la.wave < kLoadWaves)
      dma16(rs, __builtin_amdgcn_readfirstlane(mx_to + buf * 2 * kMxStage), mx_off,
            __builtin_amdgcn_readfirstlane((uint32_t)kt * kMxStage + (uint32_t)(la.wave & 1) * 1024));
  };

  if (KT > 0) load(0, 0);
  wait_loads();
  __syncthreads();
  if (KT <= 0) return;
  if (KT > 1) load(1, 1);

  MxFrags f;
  f.template read_b<0>(g_lds, g_mx_lds, 0, wm, wn, lane);
#pragma unroll
  for (int mi = 0; mi < kMI; mi++) f.read_a(g_lds, 0, mi, mi, wm, lane);
  bool pf = false;
  for (int kt = 0; kt < KT; ++kt) {
    const int buf = kt & 1;
    const char* cur = g_lds + buf * kStageBytes;
    const char* nxt = g_lds + (buf ^ 1) * kStageBytes;
    substep_mx<0>(f, cur, g_mx_lds + buf * 2 * kMxStage, 1, wm, wn, lane, acc);
    if (pf) wait_vmcnt_1();
    else wait_loads();
    __syncthreads();
    if (kt + 2 < KT) load(kt + 2, buf);
    pf = kt + kPrefetchAhead < KT &&
         prefetch_stage<mx4, true, true>(la, lb, sh, kt + kPrefetchAhead, wave, lane);
    substep_mx<1>(f, nxt, g_mx_lds + (buf ^ 1) * 2 * kMxStage, 0, wm, wn, lane, acc);
  }
}

namespace small {

// The scales of a stage's blocks: 8 bytes of K a row, 64 rows of A and then BN of B (up to 64), in 1 KiB of LDS.
// Waves 0 and 1 load A's, waves 2 and 3 B's; lanes without a row or a word of it fetch nothing and write 0 (2^-127,
// next to values that are 0).
constexpr int kScaleStage = 1024;
template <int BN> struct ScaleLoader {
  i32x4 rsrc;
  uint32_t voff, ld;
  int k0;
  uint32_t to;
  bool is_a;

  __device__ __forceinline__ void init(const uint8_t* a, uint32_t a_bytes, uint32_t lda, const uint8_t* b,
                                       uint32_t b_bytes, uint32_t ldb, int tid) {
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, row = 32 * (wave & 1) + (l >> 1);
    is_a = wave < 2;
    rsrc = is_a ? make_rsrc_words(a, a_bytes) : make_rsrc_words(b, b_bytes);
    ld = __builtin_amdgcn_readfirstlane(is_a ? lda : ldb);
    k0 = 4 * (l & 1);
    voff = is_a || row < BN ? (uint32_t)row * ld + k0 : kOob;
    to = __builtin_amdgcn_readfirstlane(wave * 256);
  }
  // a_off: A's rows start that many bytes after its descriptor's
  __device__ __forceinline__ void load(int kt, uint32_t lds, uint32_t a_off) const {
    const uint32_t k = (uint32_t)kt * 8;
    dma4(rsrc, __builtin_amdgcn_readfirstlane(lds + to), k + k0 < ld ? voff : kOob,
         __builtin_amdgcn_readfirstlane(k + (is_a ? a_off : 0u)));
  }
};

}  // namespace small
}  // namespace flce
