// MXFP4 operands in the matrix loops (flce_mx.h has the format).
#pragma once

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
