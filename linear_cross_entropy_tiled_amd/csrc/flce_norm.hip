// Layer norm of rows, forward and backward.
//
//   mean = sum x / H,  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),  xhat = (x - mean) rstd,
//   y = weight xhat + bias.
// With the upstream gradient dy and d = weight dy,
//   dx = rstd (d - sum d / H - xhat sum (d xhat) / H),
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
// Everything is formed in fp32 and rounded once to the output's type.  The variance is the
// mean of the squared distances from the mean, not a difference of two large numbers.
//
// What bounds it is memory.  Rows of up to 16384 values are held between the passes over
// them: 8 or 16 columns a thread, 64 to 1024 threads a row, and a workgroup takes row after
// row with the weight (backward: and the column sums) held too, loading the next row while
// it works on one.  Every value is read once and written once.  All of it is in registers,
// but for the backward of 8193 to 16384 columns (norm_bwd_kernel has its figures).
// N = 8192, H = 4096, bf16, fp32 parameters, where a large copy reaches 4.7 TB/s: forward
// 33 us (4.1 TB/s), backward 43 us and 5 for the parts (4.7); with 16 columns to each of 256
// threads 52, 49 and 9, as one workgroup a row with its passes from cache 196 in all.
// N = 65536, H = 2048, fp16: 108 and 156 us, 5.0 and 5.2 TB/s.
#include "flce_device.h"
#include "flce_norm.h"

namespace flce {

// VEC neighbouring values of a parameter vector of T or fp32, in pieces of up to 16 bytes (to which it is aligned).
template <typename P, int VEC> __device__ __forceinline__ void param_piece(const P* p, float* out) {
  constexpr int kMost = 16 / sizeof(P), kPiece = VEC < kMost ? VEC : kMost;
  typedef P V __attribute__((ext_vector_type(kPiece)));
#pragma unroll
  for (int k = 0; k < VEC; k += kPiece) {
    const V v = *reinterpret_cast<const V*>(p + k);
#pragma unroll
    for (int j = 0; j < kPiece; j++) out[k + j] = (float)v[j];
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void param_at(const void* p, int dtype, int i, bool in, float none, float* out) {
#pragma unroll
  for (int j = 0; j < VEC; j++) out[j] = in ? none : 0.0f;
  if (!p || !in) return;
  if (dtype == FLCE_F32) param_piece<float, VEC>(static_cast<const float*>(p) + i, out);
  else param_piece<T, VEC>(static_cast<const T*>(p) + i, out);
}

// The sum over a workgroup of 1024, on every thread.
__device__ __forceinline__ float block_sum(float v, float* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) v += lds[k];
  __syncthreads();
  return v;
}

// ---------------------------------------------------------------------------
// Rows of any length (beyond 16384): one workgroup a row, VEC columns a thread at a time; the
// passes after the first read the row from cache, the column sums read x and dy again.
// 4096 x 32768 in bf16, fp32 parameters: 164 us forward (reading and writing once takes 114),
// 337 backward (171 so); 64 x 131072 26 and 52.  By 256 threads of one column at a time 335,
// 577 and 321, 328.
// ---------------------------------------------------------------------------
template <typename T, int VEC> __global__ __launch_bounds__(1024) void norm_fwd_any_kernel(NormArgs a) {
  typedef T V __attribute__((ext_vector_type(VEC)));
  __shared__ float lds[16];
  const float inv = 1.0f / (float)a.cols;
  const int c0 = (int)threadIdx.x * VEC;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    T* y = static_cast<T*>(a.y) + r * a.cols;
    float s = 0.0f;
#pragma unroll 4
    for (int c = c0; c < a.cols; c += 1024 * VEC) {
      const V v = *reinterpret_cast<const V*>(x + c);
#pragma unroll
      for (int j = 0; j < VEC; j++) s += (float)v[j];
    }
    const float mean = block_sum(s, lds) * inv;
    s = 0.0f;
#pragma unroll 4
    for (int c = c0; c < a.cols; c += 1024 * VEC) {
      const V v = *reinterpret_cast<const V*>(x + c);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float d = (float)v[j] - mean;
        s = fmaf(d, d, s);
      }
    }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum(s, lds), inv, a.eps));
    for (int c = c0; c < a.cols; c += 1024 * VEC) {
      V v = *reinterpret_cast<const V*>(x + c);
      float w[VEC], b[VEC];
      param_at<T, VEC>(a.weight, a.param_dtype, c, true, 1.0f, w);
      param_at<T, VEC>(a.bias, a.param_dtype, c, true, 0.0f, b);
#pragma unroll
      for (int j = 0; j < VEC; j++) v[j] = (T)fmaf(((float)v[j] - mean) * rstd, w[j], b[j]);
      *reinterpret_cast<V*>(y + c) = v;
    }
    if (a.mean && threadIdx.x == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
}

template <typename T, int VEC> __global__ __launch_bounds__(1024) void norm_dx_any_kernel(NormArgs a) {
  typedef T V __attribute__((ext_vector_type(VEC)));
  __shared__ float lds[16];
  const float inv = 1.0f / (float)a.cols;
  const int c0 = (int)threadIdx.x * VEC;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + r * a.cols;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 2
    for (int c = c0; c < a.cols; c += 1024 * VEC) {
      const V v = *reinterpret_cast<const V*>(x + c), g = *reinterpret_cast<const V*>(dy + c);
      float w[VEC];
      param_at<T, VEC>(a.weight, a.param_dtype, c, true, 1.0f, w);
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const float d = (float)g[j] * w[j];
        s1 += d;
        s2 = fmaf(d, ((float)v[j] - mean) * rstd, s2);
      }
    }
    s1 = block_sum(s1, lds) * inv;
    s2 = block_sum(s2, lds) * inv;
    for (int c = c0; c < a.cols; c += 1024 * VEC) {
      V v = *reinterpret_cast<const V*>(x + c);
      const V g = *reinterpret_cast<const V*>(dy + c);
      float w[VEC];
      param_at<T, VEC>(a.weight, a.param_dtype, c, true, 1.0f, w);
#pragma unroll
      for (int j = 0; j < VEC; j++)
        v[j] = (T)(rstd * ((float)g[j] * w[j] - fmaf(((float)v[j] - mean) * rstd, s2, s1)));
      *reinterpret_cast<V*>(dx + c) = v;
    }
  }
}

// Column sums of one range of rows: 64 VEC columns by 4 threads each.
template <typename T, int VEC> __global__ __launch_bounds__(256) void norm_columns_any_kernel(NormArgs a) {
  typedef T V __attribute__((ext_vector_type(VEC)));
  __shared__ float lds[2][4][VEC][64];
  const int tid = threadIdx.x, sub = tid >> 6, lane = tid & 63, c = ((int)blockIdx.x * 64 + lane) * VEC;
  const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
  float sw[VEC], sb[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j++) sw[j] = sb[j] = 0.0f;
  if (c < a.cols) {
#pragma unroll 4
    for (int64_t r = r0 + sub; r < r1; r += 4) {
      const V g = *reinterpret_cast<const V*>(static_cast<const T*>(a.dy) + r * a.ld_dy + c);
      const V x = *reinterpret_cast<const V*>(static_cast<const T*>(a.x) + r * a.ld_x + c);
      const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        sw[j] = fmaf((float)g[j], ((float)x[j] - mean) * rstd, sw[j]);
        sb[j] += (float)g[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; j++) {
    lds[0][sub][j][lane] = sw[j];
    lds[1][sub][j][lane] = sb[j];
  }
  __syncthreads();
  if (sub >= 2 || c >= a.cols) return;
#pragma unroll
  for (int j = 0; j < VEC; j++)
    a.part[((int64_t)blockIdx.y * 2 + sub) * a.cols + c + j] =
        (lds[sub][0][j][lane] + lds[sub][1][j][lane]) + (lds[sub][2][j][lane] + lds[sub][3][j][lane]);
}

// The ranges' sums: 64 columns of dweight (blockIdx.y 0) or dbias (1), 16 threads to a column, each every 16th range.
template <typename P> __global__ __launch_bounds__(1024) void norm_parts_kernel(NormArgs a) {
  __shared__ float lds[16][64];
  void* out = blockIdx.y == 0 ? a.dw : a.db;
  if (!out) return;
  const int tid = threadIdx.x, sub = tid >> 6, c = (int)blockIdx.x * 64 + (tid & 63);
  float s = 0.0f;
  if (c < a.cols) {
    for (int p = sub; p < a.parts; p += 8 * 16) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; k++)   // eight in flight; past the last one it again, not added
        v[k] = a.part[((int64_t)min(p + 16 * k, a.parts - 1) * 2 + blockIdx.y) * a.cols + c];
#pragma unroll
      for (int k = 0; k < 8; k++) s += p + 16 * k < a.parts ? v[k] : 0.0f;
    }
  }
  lds[sub][tid & 63] = s;
  __syncthreads();
  if (sub != 0 || c >= a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) s += lds[k][tid];
  static_cast<P*>(out)[c] = (P)s;
}

// ---------------------------------------------------------------------------
// Rows in registers
// ---------------------------------------------------------------------------
// A thread's columns of a row: CPT of them in pieces of VEC, TPR threads a row.
template <typename T, int VEC, int CPT, int TPR> struct RowPart {
  static constexpr int NV = CPT / VEC;
  typedef T V __attribute__((ext_vector_type(VEC)));
  V v[NV];
  __device__ __forceinline__ static int col(int k, int t) { return (k * TPR + t) * VEC; }
  __device__ __forceinline__ void load(const T* row, int t, int cols) {
#pragma unroll
    for (int k = 0; k < NV; k++) {
      if (col(k, t) < cols) {
        v[k] = *reinterpret_cast<const V*>(row + col(k, t));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j++) v[k][j] = (T)0.0f;
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int t, int cols) const {
#pragma unroll
    for (int k = 0; k < NV; k++)
      if (col(k, t) < cols) *reinterpret_cast<V*>(row + col(k, t)) = v[k];
  }
  __device__ __forceinline__ float get(int c) const { return (float)v[c / VEC][c % VEC]; }
  __device__ __forceinline__ void set(int c, float x) { v[c / VEC][c % VEC] = (T)x; }
};

// Sums of two values over the TPR threads of a row, on each of them.  lds: [2][ROWS][TPR / 64][2]; the caller
// alternates `slot`, so that one barrier a call is enough.
template <int TPR, int ROWS>
__device__ __forceinline__ void row_sums(float& a, float& b, float* lds, int slot, int rg, int t) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a += __shfl_xor(a, o);
    b += __shfl_xor(b, o);
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* at = lds + (slot * ROWS + rg) * W * 2;
    if ((t & 63) == 0) {
      at[2 * (t >> 6)] = a;
      at[2 * (t >> 6) + 1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; w++) {
      a += at[2 * w];
      b += at[2 * w + 1];
    }
  }
}

template <typename T, int VEC, int CPT, int TPR, int ROWS>
__global__ __launch_bounds__(TPR * ROWS) void norm_fwd_kernel(NormArgs a) {
  typedef RowPart<T, VEC, CPT, TPR> Part;
  __shared__ float lds[TPR > 64 ? 4 * ROWS * (TPR / 64) : 1];
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  float w[CPT], b[CPT];
#pragma unroll
  for (int k = 0; k < Part::NV; k++) {
    const int at = Part::col(k, t);
    param_at<T, VEC>(a.weight, a.param_dtype, at, at < a.cols, 1.0f, w + k * VEC);
    param_at<T, VEC>(a.bias, a.param_dtype, at, at < a.cols, 0.0f, b + k * VEC);
  }
  const int64_t groups = (a.rows + ROWS - 1) / ROWS;
  Part next;
  next.load(static_cast<const T*>(a.x) + min((int64_t)blockIdx.x * ROWS + rg, a.rows - 1) * a.ld_x, t, a.cols);
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t r = g * ROWS + rg;
    Part x = next;
    if (g + gridDim.x < groups)
      next.load(static_cast<const T*>(a.x) + min(r + (int64_t)gridDim.x * ROWS, a.rows - 1) * a.ld_x, t, a.cols);
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; c++) s += x.get(c);
    row_sums<TPR, ROWS>(s, q, lds, 0, rg, t);
    const float mean = s * inv;
    float d[CPT];
    s = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; c++) {
      d[c] = Part::col(c / VEC, t) < a.cols ? x.get(c) - mean : 0.0f;
      s = fmaf(d[c], d[c], s);
    }
    row_sums<TPR, ROWS>(s, q, lds, 1, rg, t);
    const float rstd = 1.0f / sqrtf(fmaf(s, inv, a.eps));
#pragma unroll
    for (int c = 0; c < CPT; c++) x.set(c, fmaf(d[c] * rstd, w[c], b[c]));
    if (r < a.rows) {
      x.store(static_cast<T*>(a.y) + r * a.cols, t, a.cols);
      if (a.mean && t == 0) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
      }
    }
  }
}

// Workgroup g takes the row groups g, g + gridDim.x, ...; its column sums are part g.  512
// workgroups at most (256 of 1024 threads): each part is 8 bytes a column to write and to
// read, an eighth of the traffic at N = 8192.
// Of 8193 to 16384 columns a thread's 16 need more than the 128 registers that 1024 threads
// leave it: the weight and two column sums are 48, a row ahead of two inputs and the row in
// work 32 in 16 bits, 64 in fp32.  It spills 12 of them (16 bits, rows of whole 16 bytes; 88
// of other rows) and 72 (fp32; 81), some of which go to scratch memory and back for each row.
// 4096 rows, fp32 parameters, us here | by the kernels for any length: bf16 8200 columns 80 |
// 85, 12288 98 | 112, 16384 116 | 152, 12287 160 | 168; fp32 8200 236 | 144, 12288 262 | 224,
// 16384 297 | 306, 12287 256 | 246.  (So fp32 rows of up to some 14000 columns would be better
// off there.)
template <typename T, int VEC, int CPT, int TPR, int ROWS>
__global__ __launch_bounds__(TPR * ROWS) void norm_bwd_kernel(NormArgs a) {
  typedef RowPart<T, VEC, CPT, TPR> Part;
  __shared__ float lds[TPR > 64 ? 4 * ROWS * (TPR / 64) : 1];
  __shared__ float cs[ROWS > 1 ? TPR * CPT : 1];
  const int t = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  float w[CPT], sw[CPT], sb[CPT];
#pragma unroll
  for (int k = 0; k < Part::NV; k++) {
    const int at = Part::col(k, t);
    param_at<T, VEC>(a.weight, a.param_dtype, at, at < a.cols, 1.0f, w + k * VEC);
  }
#pragma unroll
  for (int c = 0; c < CPT; c++) sw[c] = sb[c] = 0.0f;
  const int64_t groups = (a.rows + ROWS - 1) / ROWS;
  Part xn, gn;
  float mean_n = 0.0f, rstd_n = 0.0f;
  auto load = [&](int64_t r) {
    r = min(r, a.rows - 1);
    xn.load(static_cast<const T*>(a.x) + r * a.ld_x, t, a.cols);
    gn.load(static_cast<const T*>(a.dy) + r * a.ld_dy, t, a.cols);
    mean_n = a.mean[r];
    rstd_n = a.rstd[r];
  };
  if (a.rows > 0) load((int64_t)blockIdx.x * ROWS + rg);
  int slot = 0;
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x, slot ^= 1) {
    const int64_t r = g * ROWS + rg;
    const bool here = r < a.rows;
    Part x = xn, dy = gn;
    const float mean = mean_n, rstd = rstd_n;
    if (g + gridDim.x < groups) load(r + (int64_t)gridDim.x * ROWS);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < CPT; c++) {
      const float gy = here ? dy.get(c) : 0.0f, xh = here ? (x.get(c) - mean) * rstd : 0.0f;
      const float d = gy * w[c];   // 0 past the row's end, where dy and w are
      s1 += d;
      s2 = fmaf(d, xh, s2);
      sw[c] = fmaf(gy, xh, sw[c]);
      sb[c] += gy;
    }
    if (a.dx) {
      row_sums<TPR, ROWS>(s1, s2, lds, slot, rg, t);
      s1 *= inv;
      s2 *= inv;
#pragma unroll
      for (int c = 0; c < CPT; c++)
        x.set(c, rstd * (dy.get(c) * w[c] - fmaf((x.get(c) - mean) * rstd, s2, s1)));
      if (here) x.store(static_cast<T*>(a.dx) + r * a.cols, t, a.cols);
    }
  }
  if (!a.dw && !a.db) return;
  // the row groups' sums, one after the other
  float* part = a.part + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
  for (int which = 0; which < 2; which++) {
    float* v = which == 0 ? sw : sb;
    if constexpr (ROWS > 1) {
      for (int k = ROWS - 1; k > 0; k--) {
        __syncthreads();
        if (rg == k) {
#pragma unroll
          for (int c = 0; c < CPT; c++) cs[c * TPR + t] = v[c];
        }
        __syncthreads();
        if (rg == k - 1) {
#pragma unroll
          for (int c = 0; c < CPT; c++) v[c] += cs[c * TPR + t];
        }
      }
    }
    if (rg == 0) {
#pragma unroll
      for (int c = 0; c < CPT; c++) {
        const int at = Part::col(c / VEC, t) + c % VEC;
        if (at < a.cols) part[(int64_t)which * a.cols + at] = v[c];
      }
    }
  }
}

constexpr int64_t kRegisterCols = 16384;
static int threads_per_row(int64_t cols) {   // 8 columns each, 16 beyond 8192
  int n = 64;
  while (n < 1024 && 8 * n < cols) n *= 2;
  return n;
}
static constexpr int rows_at_once(int tpr) { return tpr >= 512 ? 1 : 512 / tpr; }   // backward

int norm_parts(int64_t rows, int64_t cols) {
  if (cols > kRegisterCols) {
    const int64_t n = (rows + 31) / 32;   // up to 8192 rows at most 8 rows to a thread, beyond more
    return (int)(n < 1 ? 1 : (n > 256 ? 256 : n));
  }
  const int tpr = threads_per_row(cols), most = tpr == 1024 ? 256 : 512;
  const int64_t n = (rows + rows_at_once(tpr) - 1) / rows_at_once(tpr);
  return (int)(n < 1 ? 1 : (n > most ? most : n));
}

static size_t element_bytes(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }
static bool rows16(const void* p, int64_t ld, int dtype) {   // rows that begin on 16 bytes
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * element_bytes(dtype)) % 16 == 0;
}

template <typename T, int VEC, int CPT, int TPR>
static void norm_rows_t(const NormArgs& a, bool back, hipStream_t st) {
  if constexpr (TPR != 512 || CPT == 8) {   // (16 columns by 512 threads: forward only)
    if (back) {
      constexpr int ROWS = rows_at_once(TPR);
      norm_bwd_kernel<T, VEC, CPT, TPR, ROWS><<<a.parts, TPR * ROWS, 0, st>>>(a);
      return;
    }
  }
  constexpr int ROWS = TPR >= 256 ? 1 : 256 / TPR;
  const int64_t groups = (a.rows + ROWS - 1) / ROWS;
  norm_fwd_kernel<T, VEC, CPT, TPR, ROWS><<<(unsigned)(groups < 2048 ? groups : 2048), TPR * ROWS, 0, st>>>(a);
}

template <typename T, int VEC> static void norm_rows(const NormArgs& a, bool back, hipStream_t st) {
  switch (threads_per_row(a.cols)) {
    case 64: norm_rows_t<T, VEC, 8, 64>(a, back, st); break;
    case 128: norm_rows_t<T, VEC, 8, 128>(a, back, st); break;
    case 256: norm_rows_t<T, VEC, 8, 256>(a, back, st); break;
    case 512: norm_rows_t<T, VEC, 8, 512>(a, back, st); break;
    default:
      // (forward of 16384 x 8192 in bf16: 1024 threads of 8 columns, one workgroup a CU, 165 us; 512 of 16 102)
      if (a.cols > 8192) norm_rows_t<T, VEC, 16, 1024>(a, back, st);
      else if (back) norm_rows_t<T, VEC, 8, 1024>(a, back, st);
      else norm_rows_t<T, VEC, 16, 512>(a, back, st);
  }
}

template <typename T, int VEC> static void norm_any(const NormArgs& a, bool back, hipStream_t st) {
  const unsigned wgs = (unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20));
  if (!back) {
    norm_fwd_any_kernel<T, VEC><<<wgs, 1024, 0, st>>>(a);
    return;
  }
  if (a.rows > 0 && a.dx) norm_dx_any_kernel<T, VEC><<<wgs, 1024, 0, st>>>(a);
  if (a.dw || a.db)
    norm_columns_any_kernel<T, VEC><<<dim3((unsigned)((a.cols + 64 * VEC - 1) / (64 * VEC)), (unsigned)a.parts), 256, 0, st>>>(a);
}

template <typename T> static void norm_t(const NormArgs& a, bool back, hipStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const bool vec = rows16(a.x, a.ld_x, a.dtype) && rows16(back ? a.dx : a.y, a.cols, a.dtype) &&
                   (!back || rows16(a.dy, a.ld_dy, a.dtype)) && rows16(a.weight, 0, a.dtype) &&
                   rows16(a.bias, 0, a.dtype);
  if (a.cols > kRegisterCols) {
    if (vec) norm_any<T, kVec>(a, back, st);
    else norm_any<T, 1>(a, back, st);
    return;
  }
  if (vec) norm_rows<T, kVec>(a, back, st);
  else norm_rows<T, 1>(a, back, st);
}

static hipError_t launch_norm(const NormArgs& a, bool back, hipStream_t st) {
  if (!back && a.rows == 0) return hipSuccess;
  if (a.dtype == FLCE_BF16) norm_t<bf16>(a, back, st);
  else if (a.dtype == FLCE_F16) norm_t<f16>(a, back, st);
  else norm_t<float>(a, back, st);
  if (back && (a.dw || a.db)) {
    const dim3 grid((unsigned)((a.cols + 63) / 64), 2);
    if (a.param_dtype == FLCE_F32) norm_parts_kernel<float><<<grid, 1024, 0, st>>>(a);
    else if (a.param_dtype == FLCE_BF16) norm_parts_kernel<bf16><<<grid, 1024, 0, st>>>(a);
    else norm_parts_kernel<f16><<<grid, 1024, 0, st>>>(a);
  }
  return hipGetLastError();
}
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t st) { return launch_norm(a, false, st); }
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t st) { return launch_norm(a, true, st); }

}  // namespace flce
