// norm.cu -- residual addition, root-mean-square norm and E4M3 output in one pass.
//
// For every row, with s = x + r (r = 0 without a residual), all in binary32:
//   sum_out = round_T(s),  y = round_T(s * w / sqrt(mean(s^2) + eps)),
//   codes, scale_bytes = the 1 x 128 E4M3 quantisation of y as rounded to T,
// so that the codes are those moe_quantize_fp8 gives for y. The norm reads s
// before its rounding to T: one rounding per output. A row's sum of squares is
// held in binary32; one that overflows (|s| above about 1e17) is taken again of
// s * 2^-80, under which no row of finite values overflows and eps vanishes.
//
// A row lives in registers between its load and its stores (8-element vectors,
// vector v of the row in thread v % TPR), so x and r are read once. 16
// consecutive lanes hold the 128 columns of one scale tile.
#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kVec = 8;  // elements per vector

__device__ __forceinline__ void load8(const float* p, float (&v)[kVec]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[kVec]) {
  const uint4 raw = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[2 * j] = __low2float(h[j]), v[2 * j + 1] = __high2float(h[j]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[kVec]) {
  uint4 raw;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
  *reinterpret_cast<uint4*>(p) = raw;
}

// Sum over the TPR threads of a row, in a fixed order. `part`: the row's TPR / 32 floats.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if constexpr (TPR > 32) {
    __syncthreads();  // the previous sum's readers are done
    if ((threadIdx.x & 31) == 0) part[(threadIdx.x % TPR) >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += part[i];
  }
  return v;
}

template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) add_rmsnorm_kernel(NormArgs a) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  __shared__ float part[kRows][TPR > 32 ? TPR / 32 : 1];
  __shared__ int overflow[kRows];
  const int local = threadIdx.x / TPR, tid = threadIdx.x % TPR;
  const int vecs = a.cols / kVec;
  const T* w = static_cast<const T*>(a.w);
  const int64_t blocks = (a.rows + kRows - 1) / kRows;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {  // every thread of the block takes every turn
    const int64_t row = b * kRows + local;
    const bool live = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.res_stride : nullptr;
    float v[NV][kVec];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * TPR + tid;
      if (live && at < vecs) load8(x + at * kVec, v[i]);
    }
    if (r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = i * TPR + tid;
        if (!live || at >= vecs) continue;
        float q[kVec];
        load8(r + at * kVec, q);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] += q[j];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * TPR + tid;
      if (!live || at >= vecs) continue;
      if (a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_stride + at * kVec, v[i]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    ss = row_sum<TPR>(ss, part[local]);
    float inv = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
    // the block's rows take the second sum together: it holds a barrier
    bool big = live && !(ss < INFINITY);
    if constexpr (TPR < 128 && TPR > 32) {
      if (tid == 0) overflow[local] = big;
      __syncthreads();
      bool any = false;
#pragma unroll
      for (int i = 0; i < kRows; ++i) any |= overflow[i] != 0;
      big = any;
    }
    if (big) {
      float ss2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!live || i * TPR + tid >= vecs) continue;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float q = v[i][j] * 0x1p-80f;
          ss2 = fmaf(q, q, ss2);
        }
      }
      ss2 = row_sum<TPR>(ss2, part[local]);
      if (!(ss < INFINITY)) {
        inv = 1.0f / sqrtf(ss2 / (float)a.cols);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[i][j] *= 0x1p-80f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * TPR + tid;
      const bool on = live && at < vecs;  // with codes, uniform over each 16 lanes (cols % 128 == 0)
      float y[kVec];
      if (on) {
        if (w) {
          float q[kVec];
          load8(w + at * kVec, q);
#pragma unroll
          for (int j = 0; j < kVec; ++j) y[j] = to_f32(from_f32<T>(v[i][j] * inv * q[j]));
        } else {
#pragma unroll
          for (int j = 0; j < kVec; ++j) y[j] = to_f32(from_f32<T>(v[i][j] * inv));
        }
        if (a.y) store8(static_cast<T*>(a.y) + row * a.y_stride + at * kVec, y);
      }
      if (a.codes) {
        float m = 0.0f;
        if (on) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) m = fmaxf(m, fabsf(y[j]));
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (on) {
          const int e = ue8m0_exponent(m);
          const float sc = pow2_neg(e);
          reinterpret_cast<uint2*>(a.codes + row * a.cols)[at] =
              make_uint2(e4m3x4(y[0], y[1], y[2], y[3], sc), e4m3x4(y[4], y[5], y[6], y[7], sc));
          if ((at & 15) == 0) a.scale_bytes[row * (a.cols / 128) + (at >> 4)] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

template <typename T, int TPR, int NV>
cudaError_t launch_t(const NormArgs& a, cudaStream_t s) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  const int64_t blocks = ceil_div(a.rows, kRows);
  add_rmsnorm_kernel<T, TPR, NV><<<(unsigned)(blocks < (1 << 30) ? blocks : (1 << 30)), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int NV>
cudaError_t launch_nv(const NormArgs& a, int tpr, cudaStream_t s) {
  switch (tpr) {
    case 32: return launch_t<T, 32, NV>(a, s);
    case 64: return launch_t<T, 64, NV>(a, s);
    case 128: return launch_t<T, 128, NV>(a, s);
    case 256: return launch_t<T, 256, NV>(a, s);
    case 512: return launch_t<T, 512, NV>(a, s);
    default: return launch_t<T, 1024, NV>(a, s);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, int dtype, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.cols % kVec != 0 || a.cols > kNormMaxCols) return cudaErrorInvalidValue;
  const int vecs = a.cols / kVec;
  const bool wide = vecs <= 1024 && a.rows <= 148;
  const int per = wide ? 1 : 4;
  int tpr = 32;
  while (tpr * per < vecs) tpr *= 2;
  if (dtype == MOE_F32) return wide ? launch_nv<float, 1>(a, tpr, s) : launch_nv<float, 4>(a, tpr, s);
  return wide ? launch_nv<bf16, 1>(a, tpr, s) : launch_nv<bf16, 4>(a, tpr, s);
}

}  // namespace moe
