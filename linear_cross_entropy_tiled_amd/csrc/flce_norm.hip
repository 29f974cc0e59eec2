// Layer norm of rows, forward and backward.
//
//   mean = sum x / H,  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),  xhat = (x - mean) rstd,
//   y = weight xhat + bias.
// With the upstream gradient dy and d = weight dy,
//   dx = rstd (d - sum d / H - xhat sum (d xhat) / H),
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
// Everything is formed in fp32 and rounded once to the output's type.  The variance is the
// mean of the squared distances from the mean, not a difference of two large numbers.
#include "flce_device.h"
#include "flce_norm.h"

namespace flce {

template <typename P> __device__ __forceinline__ float param(const void* p, int i, float none) {
  return p ? (float)static_cast<const P*>(p)[i] : none;
}

// The sum over a workgroup of 256, on every thread.
__device__ __forceinline__ float block_sum(float v, float* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
  __syncthreads();
  return v;
}

// One workgroup a row, any length; the passes after the first read the row from cache.
template <typename T, typename P> __global__ __launch_bounds__(256) void norm_fwd_any_kernel(NormArgs a) {
  __shared__ float lds[4];
  const float inv = 1.0f / (float)a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    T* y = static_cast<T*>(a.y) + r * a.cols;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += 256) s += (float)x[c];
    const float mean = block_sum(s, lds) * inv;
    s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float d = (float)x[c] - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum(s, lds), inv, a.eps));
    for (int c = threadIdx.x; c < a.cols; c += 256)
      y[c] = (T)fmaf(((float)x[c] - mean) * rstd, param<P>(a.weight, c, 1.0f), param<P>(a.bias, c, 0.0f));
    if (a.mean && threadIdx.x == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
  }
}

template <typename T, typename P> __global__ __launch_bounds__(256) void norm_dx_any_kernel(NormArgs a) {
  __shared__ float lds[4];
  const float inv = 1.0f / (float)a.cols;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + r * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + r * a.cols;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float d = (float)dy[c] * param<P>(a.weight, c, 1.0f);
      s1 += d;
      s2 = fmaf(d, ((float)x[c] - mean) * rstd, s2);
    }
    s1 = block_sum(s1, lds) * inv;
    s2 = block_sum(s2, lds) * inv;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float d = (float)dy[c] * param<P>(a.weight, c, 1.0f), xhat = ((float)x[c] - mean) * rstd;
      dx[c] = (T)(rstd * (d - fmaf(xhat, s2, s1)));
    }
  }
}

// Column sums of one range of rows: 64 columns by 4 threads each.
template <typename T> __global__ __launch_bounds__(256) void norm_columns_any_kernel(NormArgs a) {
  __shared__ float lds[2][4][64];
  const int tid = threadIdx.x, sub = tid >> 6, c = (int)blockIdx.x * 64 + (tid & 63);
  const int64_t r0 = a.rows * blockIdx.y / a.parts, r1 = a.rows * (blockIdx.y + 1) / a.parts;
  float sw = 0.0f, sb = 0.0f;
  if (c < a.cols) {
    for (int64_t r = r0 + sub; r < r1; r += 4) {
      const float g = (float)static_cast<const T*>(a.dy)[r * a.ld_dy + c];
      const float xhat = ((float)static_cast<const T*>(a.x)[r * a.ld_x + c] - a.mean[r]) * a.rstd[r];
      sw = fmaf(g, xhat, sw);
      sb += g;
    }
  }
  lds[0][sub][tid & 63] = sw;
  lds[1][sub][tid & 63] = sb;
  __syncthreads();
  if (sub < 2 && c < a.cols)
    a.part[((int64_t)blockIdx.y * 2 + sub) * a.cols + c] =
        (lds[sub][0][tid & 63] + lds[sub][1][tid & 63]) + (lds[sub][2][tid & 63] + lds[sub][3][tid & 63]);
}

// The ranges' sums: 64 columns of dweight (blockIdx.y 0) or dbias (1), 16 threads to a column, each every 16th range.
template <typename P> __global__ __launch_bounds__(1024) void norm_parts_kernel(NormArgs a) {
  __shared__ float lds[16][64];
  void* out = blockIdx.y == 0 ? a.dw : a.db;
  if (!out) return;
  const int tid = threadIdx.x, sub = tid >> 6, c = (int)blockIdx.x * 64 + (tid & 63);
  float s = 0.0f;
  if (c < a.cols)
    for (int p = sub; p < a.parts; p += 16) s += a.part[((int64_t)p * 2 + blockIdx.y) * a.cols + c];
  lds[sub][tid & 63] = s;
  __syncthreads();
  if (sub != 0 || c >= a.cols) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) s += lds[k][tid];
  static_cast<P*>(out)[c] = (P)s;
}

int norm_parts(int64_t rows, int64_t) {
  const int64_t n = (rows + 31) / 32;   // 8 rows to a thread at least
  return (int)(n < 1 ? 1 : (n > 256 ? 256 : n));
}

template <typename T, typename P> static void norm_forward_t(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0) return;
  const unsigned wgs = (unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20));
  norm_fwd_any_kernel<T, P><<<wgs, 256, 0, st>>>(a);
}

template <typename T, typename P> static void norm_backward_t(const NormArgs& a, hipStream_t st) {
  const unsigned wgs = (unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20));
  if (a.rows > 0 && a.dx) norm_dx_any_kernel<T, P><<<wgs, 256, 0, st>>>(a);
  if (a.dw || a.db) {
    const unsigned n = (unsigned)((a.cols + 63) / 64);
    norm_columns_any_kernel<T><<<dim3(n, (unsigned)a.parts), 256, 0, st>>>(a);
    norm_parts_kernel<P><<<dim3(n, 2), 1024, 0, st>>>(a);
  }
}

template <typename T> static void norm_t(const NormArgs& a, bool back, hipStream_t st) {
  if (a.param_dtype == FLCE_F32) back ? norm_backward_t<T, float>(a, st) : norm_forward_t<T, float>(a, st);
  else back ? norm_backward_t<T, T>(a, st) : norm_forward_t<T, T>(a, st);
}

static hipError_t launch_norm(const NormArgs& a, bool back, hipStream_t st) {
  if (a.dtype == FLCE_BF16) norm_t<bf16>(a, back, st);
  else if (a.dtype == FLCE_F16) norm_t<f16>(a, back, st);
  else norm_t<float>(a, back, st);
  return hipGetLastError();
}
hipError_t launch_norm_forward(const NormArgs& a, hipStream_t st) { return launch_norm(a, false, st); }
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t st) { return launch_norm(a, true, st); }

}  // namespace flce
