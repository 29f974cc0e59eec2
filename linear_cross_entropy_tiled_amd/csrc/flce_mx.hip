// Quantisation to MXFP4 (flce_mx.h has the format) and back.
//
// Of a block's largest magnitude m the scale is 2^(floor(log2 m) - 2), the power that
// brings m into [4, 8), at least 2^-127; a value is rounded to the nearest code, ties to
// the even code, and to 6 beyond it.  Everything but that rounding is exact in fp32, so
// every implementation of the definition gives the same codes.  A block with NaN or an
// infinity has scale 255 (NaN) and codes 0.
#include "../../include/flce.h"
#include "flce_device.h"
#include "flce_mx.h"

namespace flce {

// A thread works on kPieces pieces of eight values, all of them in flight at once; four neighbouring lanes hold a
// block.  (Head of 128256 x 4096 in bf16: one piece a thread and comparisons in place of the conversion instruction,
// which rounds and saturates as defined, took 330 us to quantise and 285 back; 240 and 218 so, 5.5 and 6.1 TB/s.)
constexpr int kPieces = 4;

// Eight values of a block that four lanes hold: their codes, and the block's scale byte.
template <typename V> __device__ __forceinline__ uint32_t quantize_piece(const V& v, int* scale) {
  float a[8], top = 0.0f;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    a[j] = (float)v[j];
    top = fmaxf(top, fabsf(a[j]));
    bad = bad || !(fabsf(a[j]) < INFINITY);
  }
  if (bad) top = INFINITY;
  top = fmaxf(top, __shfl_xor(top, 1));
  top = fmaxf(top, __shfl_xor(top, 2));
  // the exponent field less 2; 0 (and the 2^-127 that it stands for) from there down
  const int field = (int)(__builtin_bit_cast(uint32_t, top) >> 23);
  const bool none = field == 255;
  const int code = field > 2 ? field - 2 : 0;
  *scale = none ? 255 : code;
  // to [4, 8), exactly, then to codes
  const float inv = __builtin_bit_cast(float, (uint32_t)(254 - (none ? 0 : code)) << 23);
  uint32_t out = 0;
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[0] * inv, a[1] * inv, 1.0f, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[2] * inv, a[3] * inv, 1.0f, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[4] * inv, a[5] * inv, 1.0f, 2);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[6] * inv, a[7] * inv, 1.0f, 3);
  return none ? 0u : out;
}

template <typename T> __global__ __launch_bounds__(256) void quantize_mx_kernel(const T* x, int64_t n8, uint32_t* q,
                                                                                uint8_t* scale, int words) {
  typedef T V __attribute__((ext_vector_type(8)));
  const int64_t i0 = (int64_t)blockIdx.x * (256 * kPieces) + threadIdx.x;
  V v[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; k++) v[k] = reinterpret_cast<const V*>(x)[min(i0 + k * 256, n8 - 1)];
#pragma unroll
  for (int k = 0; k < kPieces; k++) {
    const int64_t i = i0 + k * 256;
    int code;
    const uint32_t out = quantize_piece(v[k], &code);
    // four blocks' scales to a word, where all four are there
    uint32_t four = (uint32_t)code | (uint32_t)__shfl_xor(code, 4) << 8;
    four |= (uint32_t)__shfl_xor((int)four, 8) << 16;
    if (i >= n8) continue;   // whole blocks of four lanes: n8 is a multiple of 4
    q[i] = out;
    if (words && (i | 15) < n8) {
      if ((i & 15) == 0) *reinterpret_cast<uint32_t*>(scale + (i >> 2)) = four;
    } else if ((i & 3) == 0) {
      scale[i >> 2] = (uint8_t)code;
    }
  }
}

template <typename T> __global__ __launch_bounds__(256) void dequantize_mx_kernel(const uint32_t* q, const uint8_t* scale,
                                                                                  int64_t n8, T* x) {
  typedef T V __attribute__((ext_vector_type(8)));
  const int64_t i0 = (int64_t)blockIdx.x * (256 * kPieces) + threadIdx.x;
  uint32_t c[kPieces], s[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; k++) {
    const int64_t i = min(i0 + k * 256, n8 - 1);
    c[k] = q[i];
    s[k] = scale[i >> 2];
  }
#pragma unroll
  for (int k = 0; k < kPieces; k++) {
    const int64_t i = i0 + k * 256;
    if (i >= n8) return;
    // 2^(s - 127): below the normal numbers for s = 0
    const float f = s[k] == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, s[k] == 0 ? 1u << 22 : s[k] << 23);
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 1),
                p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.0f, 3);
    const float y[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    V v;
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = (T)(y[j] * f);
    reinterpret_cast<V*>(x)[i] = v;
  }
}

constexpr int64_t kMostGroups = int64_t(1) << 22;   // of 256 threads: a launch of 2^32 threads or more leaves some out
constexpr int64_t kGroup = 256 * kPieces;

template <typename T> static void quantize_t(const void* x, int64_t n8, uint8_t* q, uint8_t* scale, hipStream_t st) {
  const int words = (reinterpret_cast<uintptr_t>(scale) & 3) == 0;
  for (int64_t i = 0; i < n8; i += kMostGroups * kGroup) {
    const int64_t n = n8 - i < kMostGroups * kGroup ? n8 - i : kMostGroups * kGroup;
    quantize_mx_kernel<T><<<(unsigned)((n + kGroup - 1) / kGroup), 256, 0, st>>>(
        static_cast<const T*>(x) + i * 8, n, reinterpret_cast<uint32_t*>(q) + i, scale + i / 4, words);
  }
}
template <typename T> static void dequantize_t(const uint8_t* q, const uint8_t* scale, int64_t n8, void* x, hipStream_t st) {
  for (int64_t i = 0; i < n8; i += kMostGroups * kGroup) {
    const int64_t n = n8 - i < kMostGroups * kGroup ? n8 - i : kMostGroups * kGroup;
    dequantize_mx_kernel<T><<<(unsigned)((n + kGroup - 1) / kGroup), 256, 0, st>>>(
        reinterpret_cast<const uint32_t*>(q) + i, scale + i / 4, n, static_cast<T*>(x) + i * 8);
  }
}

hipError_t launch_quantize_mx(int dtype, const void* x, int64_t blocks, uint8_t* q, uint8_t* scale, hipStream_t st) {
  if (dtype == FLCE_BF16) quantize_t<bf16>(x, 4 * blocks, q, scale, st);
  else if (dtype == FLCE_F16) quantize_t<f16>(x, 4 * blocks, q, scale, st);
  else quantize_t<float>(x, 4 * blocks, q, scale, st);
  return hipGetLastError();
}
hipError_t launch_dequantize_mx(int dtype, const uint8_t* q, const uint8_t* scale, int64_t blocks, void* x,
                                hipStream_t st) {
  if (dtype == FLCE_BF16) dequantize_t<bf16>(q, scale, 4 * blocks, x, st);
  else if (dtype == FLCE_F16) dequantize_t<f16>(q, scale, 4 * blocks, x, st);
  else dequantize_t<float>(q, scale, 4 * blocks, x, st);
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void pad_scales_kernel(const uint8_t* scale, int64_t rows, int cols, int ld, uint8_t* out) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < ld; c += 256) out[r * ld + c] = c < cols ? scale[r * cols + c] : 0;
}
hipError_t launch_pad_scales(const uint8_t* scale, int64_t rows, int cols, int ld, uint8_t* out, hipStream_t st) {
  if (rows > 0) pad_scales_kernel<<<(unsigned)(rows < 65536 ? rows : 65536), 256, 0, st>>>(scale, rows, cols, ld, out);
  return hipGetLastError();
}

// 64 rows (number `unit`) by 16 stages (128 blocks) a workgroup, through LDS; weight: layout a, else b.
__device__ __forceinline__ void tile_scales(const uint8_t* scales, int64_t rows, int ld, int stages, bool weight, int unit,
                                            int chunk, uint8_t* to, uint32_t (&lds)[64][33]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const int i = k * 256 + tid, r = i >> 5, c = (i & 31) * 4 + chunk * 128;
    const int64_t row = (int64_t)unit * 64 + r;
    lds[r][i & 31] = row < rows && c < ld ? *reinterpret_cast<const uint32_t*>(scales + row * ld + c) : 0u;
  }
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(to) + (int64_t)(unit >> 2) * stages * (kMxStage / 4);
  auto scale = [&](int row, int block) { return (lds[row][block >> 2] >> (8 * (block & 3))) & 255u; };
#pragma unroll
  for (int k = 0; k < 8; k++) {
    // a stage's 128 words of these 64 rows: two halves of a's words, or two words of b
    const int i = k * 256 + tid, stage = i >> 7, kt = chunk * 16 + stage, lane = (i >> 1) & 63;
    if (kt >= stages) continue;
    const int p = i & 1;
    if (weight) {
      // two sub-steps' halves, 32 rows each: bytes 2 (unit % 2) and up of the words
      const int half = unit & 1, sub = (unit >> 1) & 1;
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int s = 2 * p + j, block = 8 * stage + 2 * s + (lane >> 5);
        const uint32_t v = scale(lane & 31, block) | scale(32 + (lane & 31), block) << 8;
        reinterpret_cast<uint16_t*>(out + (int64_t)kt * 512 + sub * 256 + lane * 4 + s)[half] = (uint16_t)v;
      }
    } else {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; j++)
        v |= scale(32 * (j & 1) + (lane & 31), 8 * stage + 2 * (2 * p + (j >> 1)) + (lane >> 5)) << (8 * j);
      out[(int64_t)kt * 512 + (unit & 3) * 128 + lane * 2 + p] = v;
    }
  }
}

// Workgroups from 0: kPieces pieces a thread of the hidden states' rows, padded to whole tiles with scales of 0 (their
// codes, past the last row and block, are loaded as 0).  From n_quantise: the scales' order.
struct MxPrepArgs {
  MxPrep p;
  int64_t pieces;              // of padded rows
  int row_blocks;              // blocks of a padded row
  int n_quantise, w_units, chunks;
};
template <typename T> __global__ __launch_bounds__(256) void mx_prep_kernel(MxPrepArgs a) {
  __shared__ uint32_t lds[64][33];
  const MxPrep& p = a.p;
  if ((int)blockIdx.x >= a.n_quantise) {
    const int id = (int)blockIdx.x - a.n_quantise, chunk = id % a.chunks, unit = id / a.chunks;
    if (unit < a.w_units) tile_scales(p.w_scale, p.w_rows, p.ld, p.stages, true, unit, chunk, p.w_out, lds);
    else tile_scales(p.h_scale, p.n, p.ld, p.stages, false, unit - a.w_units, chunk, p.h_out, lds);
    return;
  }
  typedef T V __attribute__((ext_vector_type(8)));
  const int64_t i0 = (int64_t)blockIdx.x * kGroup + threadIdx.x;
  int64_t row[kPieces];
  int block[kPieces];
  V v[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; k++) {
    const int64_t b = (i0 + 256 * k) >> 2;
    row[k] = b < (int64_t(1) << 32) ? (int64_t)((uint32_t)b / (uint32_t)a.row_blocks) : b / a.row_blocks;
    block[k] = (int)(b - row[k] * a.row_blocks);
    const bool here = row[k] < p.n && block[k] < p.blocks;
#pragma unroll
    for (int j = 0; j < 8; j++) v[k][j] = (T)0.0f;
    if (here) v[k] = reinterpret_cast<const V*>(p.x)[(row[k] * p.blocks + block[k]) * 4 + (threadIdx.x & 3)];
  }
#pragma unroll
  for (int k = 0; k < kPieces; k++) {
    int code;
    const uint32_t out = quantize_piece(v[k], &code);
    if (i0 + 256 * k >= a.pieces) continue;
    const int b = block[k];
    const int64_t r = row[k];
    if (r < p.n && b < p.blocks)
      reinterpret_cast<uint32_t*>(p.q)[(r * p.blocks + b) * 4 + (threadIdx.x & 3)] = out;
    if ((threadIdx.x & 3) != 0) continue;
    if (r < p.n && b < p.ld) p.scale[r * p.ld + b] = (uint8_t)code;
    if (p.stages > 0) {
      const int s = (b >> 1) & 3, lane = (int)(r & 31) + 32 * (b & 1);
      p.h_out[((r >> 8) * p.stages + (b >> 3)) * kMxStage + ((r >> 6) & 3) * 512 + lane * 8 + (s >> 1) * 4 + (s & 1) * 2 +
              ((r >> 5) & 1)] = (uint8_t)code;
    }
  }
}

hipError_t launch_mx_prep(int dtype, const MxPrep& p, hipStream_t st) {
  MxPrepArgs a{};
  a.p = p;
  a.chunks = (p.stages + 15) / 16;
  int64_t rows = 0;
  if (p.x) {
    a.row_blocks = p.stages > 0 ? p.stages * 8 : p.ld;
    rows = p.stages > 0 ? (int64_t)p.h_tiles * 256 : p.n;
  }
  a.pieces = rows * a.row_blocks * 4;
  a.n_quantise = (int)((a.pieces + kGroup - 1) / kGroup);
  a.w_units = p.stages > 0 ? p.w_tiles * 4 : 0;
  const int units = a.w_units + (p.stages > 0 && !p.x ? p.h_tiles * 4 : 0);
  const int64_t wgs = a.n_quantise + (int64_t)units * a.chunks;
  if (wgs == 0) return hipSuccess;
  if (dtype == FLCE_BF16) mx_prep_kernel<bf16><<<(unsigned)wgs, 256, 0, st>>>(a);
  else if (dtype == FLCE_F16) mx_prep_kernel<f16><<<(unsigned)wgs, 256, 0, st>>>(a);
  else mx_prep_kernel<float><<<(unsigned)wgs, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace flce
