// 4-bit microscaled operands (MXFP4): the type's tag, matrix instruction and launchers (internal).
//
// 32 neighbouring values of a row share one power of two, held as a byte s (2^(s - 127),
// 255 = NaN); each value is a 4-bit code, sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (two
// to a byte, the earlier one in the low half).  A lane's 16 bytes of K are exactly one such
// block: v_mfma_scale_f32_16x16x128_f8f6f4 takes them as the 8- and 16-bit instructions take
// theirs, and the block's scale byte in a register of its own.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace flce {

struct mx4 {   // one byte: two values
  uint8_t two;
};

template <typename T> inline constexpr bool is_mx = false;
template <> inline constexpr bool is_mx<mx4> = true;

hipError_t launch_quantize_mx(int dtype, const void* x, int64_t blocks, uint8_t* q, uint8_t* scale, hipStream_t st);
hipError_t launch_dequantize_mx(int dtype, const uint8_t* q, const uint8_t* scale, int64_t blocks, void* x,
                                hipStream_t st);
// Scale rows of `cols` bytes to rows of `ld` bytes, a multiple of 4.
hipError_t launch_pad_scales(const uint8_t* scale, int64_t rows, int cols, int ld, uint8_t* out, hipStream_t st);
// Scales (rows of ld bytes, a multiple of 4; 0 past the last row and block) in the order of the large tiles, which
// take six words a lane and stage from LDS for all their matrix instructions' scales (one byte a fragment out of
// rows as they are stored would be 24 reads).  A stage is 256 values, 8 blocks, four sub-steps s of 2; lane l holds
// row l % 32 and block 2 s + l / 32.  Of a tile of 256 rows and a stage, kMxStage bytes:
//  a (the weight):        for each 128 rows and lane four words, by s; byte m is row 32 m + l % 32;
//  b (the hidden states): for each 64 rows and lane two words; byte 2 (s % 2) + n of word s / 2 is row 32 n + l % 32.
// Both in one launch.
constexpr int kMxStage = 2048;
// What a call's matrix kernels read, made in one launch: the hidden states' codes and scales where x is given (rows of
// ld scale bytes, as the small tiles take them), and with `stages` the scales in the large tiles' order.
struct MxPrep {
  int64_t n;                   // hidden states
  int blocks, ld, stages;      // of a row; scale bytes from row to row (a multiple of 4); 0 stages: no large tiles
  int w_tiles, h_tiles;        // large tiles of 256 rows
  const void* x;               // hidden states to quantise, or NULL
  uint8_t* q;
  uint8_t* scale;
  const uint8_t* w_scale;      // the weight's, rows of ld bytes
  int64_t w_rows;
  const uint8_t* h_scale;      // the hidden states' where x is NULL
  uint8_t* w_out;
  uint8_t* h_out;
};
hipError_t launch_mx_prep(int dtype, const MxPrep& p, hipStream_t st);

}  // namespace flce
