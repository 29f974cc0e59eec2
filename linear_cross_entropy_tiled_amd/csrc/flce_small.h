// Small-tile matrix loop, for problems that give the 256 x 256 loop of
// flce_device.h too few tiles for the chip: C[64 x BN] += A[64 x K] . B[BN x K]^T
// by 4 waves, BN 64 (2 x 2 waves of 32 x 32), 32 (2 x 2 waves of 32 x 16; MXFP4 only) or 16 (4 x 1 waves of 16 x 16).
//
// Operands, fragments and accumulator layout are those of the large loop (stages of
// 128 bytes of K per row, K-major or M/N-major); n stage buffers keep n - 1 stages of
// loads in flight under one barrier a stage, and several workgroups share a CU.  A 64 x 64
// tile reads its fragments twice as often per matrix operation as the large tile, which
// costs the 16-bit types about half their rate and fp32, whose matrix instructions take
// 16 times as long per byte, nothing.
#pragma once

#include "flce_device.h"
#include "flce_mx_device.h"

namespace flce {
namespace small {

constexpr int kBMs = 64;
constexpr int kThreadsS = 256;
constexpr int kStageA = kBMs * kBKB;                             // 8 KiB
// Stage buffers: three at BN 64 (48 KiB), so that three workgroups share a CU; two for
// fp32 there, whose stage takes 1024 cycles of matrix instructions, and where a fourth
// workgroup is worth 5%.  Four at BN 16 (40 KiB, 42 with the sides), three workgroups as
// well: 4 tokens at V = 128256 in 8 bits took 114 us, with three buffers 136, with five
// within 2% of four.
template <typename T> constexpr int stages(int bn) { return bn <= 32 ? 4 : (sizeof(T) == 4 ? 2 : 3); }
constexpr int stage_bytes(int bn) { return (kBMs + bn) * kBKB; }
template <typename T> constexpr int lds_bytes(int bn) { return stages<T>(bn) * stage_bytes(bn); }

template <int BN> struct Shape {
  static constexpr int WM = BN == 16 ? 4 : 2, WN = 4 / WM;       // waves
  static constexpr int MI = kBMs / 16 / WM, NI = BN / 16 / WN;   // 16 x 16 tiles per wave
};

// Direct-to-LDS loads of one operand's stages: block b (1 KiB of the stage, 8 rows of
// 128 bytes, or for fp32 M/N-major 4 rows of 256) is loaded by wave b / PER.
template <typename T, bool KMAJOR, int ROWS> struct Loader {
  static constexpr int BLOCKS = ROWS * kBKB / 1024;
  static constexpr int PER = BLOCKS >= 4 ? BLOCKS / 4 : 1;       // blocks of a loading wave
  i32x4 rsrc;
  uint32_t voff[PER];
  int kc[PER];
  int k_bytes;
  uint32_t ld;
  int first;      // the wave's first block
  bool loads;     // whether the wave has any

  __device__ __forceinline__ void init(const OperandDesc& d, int tid) {
    rsrc = make_rsrc_words(d.base, d.nrec);
    k_bytes = __builtin_amdgcn_readfirstlane(d.k_bytes);
    ld = __builtin_amdgcn_readfirstlane(d.ld_bytes);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
    first = wave * PER;
    loads = first < BLOCKS;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int b = first + i;
      if constexpr (KMAJOR) {
        // as in OperandLoader: chunk c of row r at slot c ^ ((r >> 1) & 7)
        kc[i] = 16 * ((l & 7) ^ ((4 * b + (l >> 4)) & 7));
        voff[i] = (uint32_t)(8 * b + (l >> 3)) * d.ld_bytes + kc[i];
      } else if constexpr (sizeof(T) == 2) {
        // K row r (64 elements, 8 chunks): chunk c at slot c ^ 2 f, f = bits 1 and 3 of r
        const int r = 8 * b + (l >> 3), f = ((r >> 1) & 1) | (((r >> 3) & 1) << 1);
        const int c = (l & 7) ^ (2 * f);
        kc[i] = 0;
        voff[i] = 8 * c < d.cols_valid ? (uint32_t)r * d.ld_bytes + 16 * c : kOob;
      } else {
        // fp32 K row r (64 elements, 16 chunks): chunk c at slot c ^ 4 ((r >> 2) & 3)
        const int r = 4 * b + (l >> 4), c = (l & 15) ^ (4 * (b & 3));
        kc[i] = 0;
        voff[i] = 4 * c < d.cols_valid ? (uint32_t)r * d.ld_bytes + 16 * c : kOob;
      }
    }
  }

  // (K-major: rows starting `row_off` bytes after the descriptor's)
  __device__ __forceinline__ void load(int kt, uint32_t lds, uint32_t row_off = 0) const {
    if (!loads) return;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      if constexpr (KMAJOR) {
        const uint32_t k0 = (uint32_t)kt * kBKB;
        dma16(rsrc, __builtin_amdgcn_readfirstlane(lds + (first + i) * 1024),
              (int)k0 + kc[i] < k_bytes ? voff[i] : kOob, __builtin_amdgcn_readfirstlane(k0 + row_off));
      } else {
        dma16(rsrc, __builtin_amdgcn_readfirstlane(lds + (first + i) * 1024), voff[i],
              (uint32_t)kt * (kBKB / sizeof(T)) * ld);
      }
    }
  }
};

// Fragments: K-major as in the large loop; M/N-major with the row lengths above.
template <typename T, bool KMAJOR> struct Frags : Frag<T, KMAJOR> {};
template <typename V8> struct Frags16MN {
  typedef V8 type;
  // see Frag16MN.  Rows are 128 bytes, two to a line of all banks: the eight rows that
  // two lane groups read at once differ in bits 0, 1 and 3; bit 0 picks the half of the
  // line and bits 1 and 3 (f) the quarter of the row.
  __device__ __forceinline__ static type read(const char* op, int c0, int s, int lane) {
    const int g = lane >> 4, a = lane & 15;
    const int row = 32 * s + 8 * g + (a >> 2);
    const int u = (c0 >> 2) + (a & 3);
    const int f0 = ((row >> 1) & 1) | (((row >> 3) & 1) << 1);   // row + 4 has the same bits 1 and 3
    const int off = row * 128 + ((u ^ (f0 << 2)) << 3);
    i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)(op + off));
    i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4*)(op + off + 4 * 128));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    i16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(V8, v);
  }
};
template <> struct Frags<bf16, false> : Frags16MN<bf16x8> {};
template <> struct Frags<f16, false> : Frags16MN<f16x8> {};
template <> struct Frags<float, false> {
  typedef f32x4 type;
  __device__ __forceinline__ static type read(const char* op, int c0, int s, int lane) {
    const int col = c0 + (lane & 15);
    const int k0 = (4 * s + (lane >> 4)) * 4;   // (k0 >> 2) & 3 = lane >> 4: the four groups read four quarters
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int slot = (col >> 2) ^ (4 * ((k0 >> 2) & 3));
      v[j] = *reinterpret_cast<const float*>(op + (k0 + j) * 256 + slot * 16 + (col & 3) * 4);
    }
    return v;
  }
};

template <int N> __device__ __forceinline__ void wait_vmcnt() {
  static_assert(N <= 15, "the high bits of vmcnt are not set here");
  __builtin_amdgcn_s_waitcnt(0x0F70 | N);
}

// One stage's matrix instructions.
template <typename T, bool A_KMAJOR, bool B_KMAJOR, int BN>
__device__ __forceinline__ void stage_mma(const char* st, int wm, int wn, int lane,
                                          Acc (&acc)[Shape<BN>::MI][Shape<BN>::NI]) {
  typedef Shape<BN> S;
#pragma unroll
  for (int s = 0; s < kSubsteps; s++) {
    typename Frags<T, A_KMAJOR>::type a[S::MI];
    typename Frags<T, B_KMAJOR>::type b[S::NI];
#pragma unroll
    for (int mi = 0; mi < S::MI; mi++) a[mi] = Frags<T, A_KMAJOR>::read(st, (wm * S::MI + mi) * 16, s, lane);
#pragma unroll
    for (int ni = 0; ni < S::NI; ni++)
      b[ni] = Frags<T, B_KMAJOR>::read(st + kStageA, (wn * S::NI + ni) * 16, s, lane);
#pragma unroll
    for (int mi = 0; mi < S::MI; mi++)
#pragma unroll
      for (int ni = 0; ni < S::NI; ni++) mma(acc[mi][ni], a[mi], b[ni]);
  }
}

// The same of MXFP4 operands; sc: the stage's scales.
template <int BN>
__device__ __forceinline__ void stage_mma_mx(const char* st, const char* sc, int wm, int wn, int lane,
                                             Acc (&acc)[Shape<BN>::MI][Shape<BN>::NI]) {
  typedef Shape<BN> S;
  const uint8_t* row = reinterpret_cast<const uint8_t*>(sc) + 8 * (lane & 15) + (lane >> 4);
#pragma unroll
  for (int s = 0; s < kSubsteps; s++) {
    i32x4 a[S::MI], b[S::NI];
    int sa[S::MI], sb[S::NI];
#pragma unroll
    for (int mi = 0; mi < S::MI; mi++) {
      a[mi] = Frag<mx4, true>::read(st, (wm * S::MI + mi) * 16, s, lane);
      sa[mi] = row[(wm * S::MI + mi) * 128 + 4 * s];
    }
#pragma unroll
    for (int ni = 0; ni < S::NI; ni++) {
      b[ni] = Frag<mx4, true>::read(st + kStageA, (wn * S::NI + ni) * 16, s, lane);
      sb[ni] = row[512 + (wn * S::NI + ni) * 128 + 4 * s];
    }
#pragma unroll
    for (int mi = 0; mi < S::MI; mi++)
#pragma unroll
      for (int ni = 0; ni < S::NI; ni++) mma_mx<0, 0>(acc[mi][ni], a[mi], b[ni], sa[mi], sb[ni]);
  }
}

// Waits until at most the loads of `later` stages are outstanding (a wave that has issued
// others since waits for a little more).
template <typename T, bool A_KMAJOR, bool B_KMAJOR, int BN, int LATER>
__device__ __forceinline__ void wait_stage(bool b_loads) {
  constexpr int A = Loader<T, A_KMAJOR, kBMs>::PER + (is_mx<T> ? 1 : 0), B = Loader<T, B_KMAJOR, BN>::PER;
  if (b_loads) wait_vmcnt<LATER * (A + B)>();
  else wait_vmcnt<LATER * A>();
}

// run(from, to, acc) for the stages 0 to KT.  fp32 products are summed 512 at a time and the
// sums added up: one chain of K / 4 matrix instructions would round every one at the size of
// the whole sum (a tenth to a quarter off the error of log p at H = 1024 to 2048, for 1 to 2%
// of the time).  Forward and backward sum alike, so that a row's softmax keeps adding up to 1.
template <typename T, int BN, typename F>
__device__ __forceinline__ void in_blocks(int KT, Acc (&acc)[Shape<BN>::MI][Shape<BN>::NI], F&& run) {
  if constexpr (sizeof(T) == 4) {
    constexpr int kBlock = 16;
    for (int kt = 0; kt < KT; kt += kBlock) {
      Acc part[Shape<BN>::MI][Shape<BN>::NI];
#pragma unroll
      for (int mi = 0; mi < Shape<BN>::MI; mi++)
#pragma unroll
        for (int ni = 0; ni < Shape<BN>::NI; ni++) part[mi][ni] = Acc{0.0f, 0.0f, 0.0f, 0.0f};
      run(kt, min(kt + kBlock, KT), part);
#pragma unroll
      for (int mi = 0; mi < Shape<BN>::MI; mi++)
#pragma unroll
        for (int ni = 0; ni < Shape<BN>::NI; ni++) acc[mi][ni] += part[mi][ni];
    }
  } else {
    run(0, KT, acc);
  }
}

// The loop.  lds: lds_bytes<T>(BN).  No load is in flight and every wave has
// passed its last LDS read when it returns after the caller's next barrier; acc must be
// zeroed by the caller.
template <typename T, bool A_KMAJOR, bool B_KMAJOR, int BN>
__device__ __forceinline__ void mainloop(const OperandDesc& da, const OperandDesc& db, int KT, char* lds,
                                         Acc (&acc)[Shape<BN>::MI][Shape<BN>::NI]) {
  typedef Shape<BN> S;
  constexpr int SB = stage_bytes(BN), kStages = stages<T>(BN);
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  Loader<T, A_KMAJOR, kBMs> la;
  Loader<T, B_KMAJOR, BN> lb;
  la.init(da, tid);
  lb.init(db, tid);
  const uint32_t base = lds_addr_of(lds);
#pragma unroll
  for (int p = 0; p < kStages - 1; p++)
    if (p < KT) {
      la.load(p, base + p * SB);
      lb.load(p, base + p * SB + kStageA);
    }
  int buf = 0;
  in_blocks<T, BN>(KT, acc, [&](int kt, int end, Acc (&to)[S::MI][S::NI]) {
    for (; kt < end; ++kt) {
      // stage kt has landed when at most the later stages' loads are outstanding
      if (kt + kStages - 2 < KT) wait_stage<T, A_KMAJOR, B_KMAJOR, BN, kStages - 2>(lb.loads);
      else wait_loads();
      __syncthreads();   // and every wave has read stage kt - 1, whose buffer is loaded next
      if (kt + kStages - 1 < KT) {
        const int nb = buf == 0 ? kStages - 1 : buf - 1;
        la.load(kt + kStages - 1, base + nb * SB);
        lb.load(kt + kStages - 1, base + nb * SB + kStageA);
      }
      stage_mma<T, A_KMAJOR, B_KMAJOR, BN>(lds + buf * SB, wm, wn, lane, to);
      buf = buf == kStages - 1 ? 0 : buf + 1;
    }
  });
}

}  // namespace small
}  // namespace flce
