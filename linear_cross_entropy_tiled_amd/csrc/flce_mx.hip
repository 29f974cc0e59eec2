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
// which rounds and saturates as defined, took 330 us to quantise and 285 back.)
constexpr int kPieces = 4;

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
    float a[8], top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      a[j] = (float)v[k][j];
      top = fmaxf(top, fabsf(a[j]));
      bad = bad || !(fabsf(a[j]) < INFINITY);
    }
    if (bad) top = INFINITY;
    top = fmaxf(top, __shfl_xor(top, 1));
    top = fmaxf(top, __shfl_xor(top, 2));
    // the exponent field less 2; 0 (and the 2^-127 that it stands for) from there down
    const int field = (int)(__builtin_bit_cast(uint32_t, top) >> 23);
    const bool none = field == 255;
    const int code = none ? 255 : (field > 2 ? field - 2 : 0);
    // to [4, 8), exactly, then to codes
    const float inv = __builtin_bit_cast(float, (uint32_t)(254 - (none ? 0 : code)) << 23);
    uint32_t out = 0;
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[0] * inv, a[1] * inv, 1.0f, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[2] * inv, a[3] * inv, 1.0f, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[4] * inv, a[5] * inv, 1.0f, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, a[6] * inv, a[7] * inv, 1.0f, 3);
    if (none) out = 0;
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

// 64 rows by 16 stages (128 blocks) a workgroup, through LDS.
struct MxTileArgs {
  MxTiles t[2];
  int ld, stages, chunks;   // chunks of 16 stages
};
__global__ __launch_bounds__(256) void mx_tile_kernel(MxTileArgs a) {
  __shared__ uint32_t lds[64][33];
  const int per_first = a.t[0].tiles * 4 * a.chunks;
  const int which = (int)blockIdx.x >= per_first, id = (int)blockIdx.x - (which ? per_first : 0);
  const MxTiles t = a.t[which];
  const int chunk = id % a.chunks, unit = id / a.chunks;   // unit: 64 rows
  const int tid = threadIdx.x;
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const int i = k * 256 + tid, r = i >> 5, c = (i & 31) * 4 + chunk * 128;
    const int64_t row = (int64_t)unit * 64 + r;
    lds[r][i & 31] = row < t.rows && c < a.ld ? *reinterpret_cast<const uint32_t*>(t.scale + row * a.ld + c) : 0u;
  }
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(t.out) + (int64_t)(unit >> 2) * a.stages * (kMxStage / 4);
  auto scale = [&](int row, int block) { return (lds[row][block >> 2] >> (8 * (block & 3))) & 255u; };
#pragma unroll
  for (int k = 0; k < 8; k++) {
    // a stage's 128 words of these 64 rows: two halves of a's words, or two words of b
    const int i = k * 256 + tid, stage = i >> 7, kt = chunk * 16 + stage, lane = (i >> 1) & 63;
    if (kt >= a.stages) continue;
    if (which == 0) {
      // two sub-steps' halves, 32 rows each: bytes 2 (unit % 2) and up of the words
      const int p = i & 1, half = unit & 1, sub = (unit >> 1) & 1;
#pragma unroll
      for (int q = 0; q < 2; q++) {
        const int s = 2 * p + q, block = 8 * stage + 2 * s + (lane >> 5);
        const uint32_t v = scale(lane & 31, block) | scale(32 + (lane & 31), block) << 8;
        reinterpret_cast<uint16_t*>(out + (int64_t)kt * 512 + sub * 256 + lane * 4 + s)[half] = (uint16_t)v;
      }
    } else {
      const int p = i & 1;
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; j++)
        v |= scale(32 * (j & 1) + (lane & 31), 8 * stage + 2 * (2 * p + (j >> 1)) + (lane >> 5)) << (8 * j);
      out[(int64_t)kt * 512 + (unit & 3) * 128 + lane * 2 + p] = v;
    }
  }
}
hipError_t launch_tile_scales(const MxTiles& a, const MxTiles& b, int ld, int stages, hipStream_t st) {
  MxTileArgs m;
  m.t[0] = a;
  m.t[1] = b;
  m.ld = ld;
  m.stages = stages;
  m.chunks = (stages + 15) / 16;
  mx_tile_kernel<<<(unsigned)((a.tiles + b.tiles) * 4 * m.chunks), 256, 0, st>>>(m);
  return hipGetLastError();
}

}  // namespace flce
