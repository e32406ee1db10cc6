// norm.cu -- residual addition, root-mean-square norm and E4M3 output in one pass.
//
// For every row, with s = x + r (r = 0 without a residual), all in binary32:
//   sum_out = round_T(s),  y = round_T(s * w / sqrt(mean(s^2) + eps)),
//   codes, scale_bytes = the 1 x 128 E4M3 quantisation of y as rounded to T,
// so that the codes are those moe_quantize_fp8 gives for y. The norm reads s
// before its rounding to T. A row's sum of squares is
// held in binary32; where the mean square overflows (|s| above about 1e17), or it and eps
// nearly vanish (below 2^-100), it is taken again of s times a power of two (norm_of).
//
// A row lives in registers between its loads and its stores, as the raw vectors of x and r (8
// elements, vector v of the row in thread v % TPR), so each is read once and all of a row's loads
// are in flight together; s is formed twice. 16 consecutive lanes hold the 128 columns of one scale
// tile.
#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kVec = 8;  // elements per vector
constexpr int kFewRows = 148;

// Eight elements as loaded. x and r bypass L1 (they may be the call's outputs, and the weight stays there).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
};
template <>
struct Raw<bf16> {
  uint4 a;
};
__device__ __forceinline__ void load8(Raw<float>& r, const float* p) {
  r.a = __ldcg(reinterpret_cast<const float4*>(p));
  r.b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void load8(Raw<bf16>& r, const bf16* p) { r.a = __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void load8_weight(Raw<float>& r, const float* p) {
  r.a = __ldg(reinterpret_cast<const float4*>(p));
  r.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
__device__ __forceinline__ void load8_weight(Raw<bf16>& r, const bf16* p) { r.a = __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void values(const Raw<float>& r, float (&v)[kVec]) {
  v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w, v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void values(const Raw<bf16>& r, float (&v)[kVec]) {
  const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
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

// y = s * scale * (inv + inv_lo) (* w): scale is 1, or 2^-8 for a row whose mean square overflows.
struct Norm {
  float scale, inv, inv_lo;
};

// 1 / sqrt(ss / cols + eps) to about twice binary32's precision: an approximation and one Newton
// step whose residual 1 - a inv^2 is formed by fused multiply-adds. With the product of a value
// compensated too (finish_vector), what is rounded in front of the value itself is s and the sum of
// squares, and a bf16 value goes through binary32. Rows whose sum is exact give binary32 values rounded
// once; of 4096 x 5120 normal ones 34 % differ from the exact norm rounded once, by the sum's roundings,
// against 51 % with three rounded products. Of 29 million bf16 values 223 differ, nearly all by the
// rounding of s = x + r to binary32 where x and r are far apart. (The sum of squares with its remainder
// carried along would leave 202, and takes 4 to 18 % longer.)
__device__ __forceinline__ Norm inverse_rms(float ss, const NormArgs& n, float eps) {
  const float q = ss * n.inv_cols, q_lo = fmaf(-q, (float)n.cols, ss) * n.inv_cols;
  const float a = q + eps, z = a - q;
  const float a_lo = ((q - (a - z)) + (eps - z)) + q_lo;
  const float inv = rsqrtf(a), p = inv * inv;
  const float r = fmaf(-a, p, 1.0f) - a * fmaf(inv, inv, -p) - a_lo * p;
  // (r means nothing where a is infinite, or so small that p overflows)
  return Norm{1.0f, inv, a >= 0x1p-120f && a < INFINITY ? 0.5f * inv * r : 0.0f};
}

// The row's Norm. square_sum(scale, store) sums (s * scale)^2 over the row (and stores sum_out).
// Where the mean square with eps overflows, the root is that of s * 2^-80 and eps * 2^-160: its inverse lies in
// [2^-48, 2^24], and of the 2^-80 that takes it back 2^-72 go to it and 2^-8 to s, so that neither leaves
// binary32's range: 2^-80 times s alone took the digits of values below 2^-46 beside others above 1e17.
// Where mean square and eps are below 2^-100, the squares vanish or lose digits: the root is that of s * 2^80 and
// eps * 2^160, its inverse below 2^-5, and all of the 2^80 goes to it.
template <int TPR, int ROWS, typename Sum>
__device__ __forceinline__ Norm norm_of(const NormArgs& a, bool live, int local, int tid, int* overflow, Sum square_sum) {
  const float ss = square_sum(1.0f, true);
  Norm n = inverse_rms(ss, a, a.eps);
  // the block's rows take the second sum together: it holds a barrier
  const bool tiny = n.inv > 0x1p50f, mine = live && (tiny || !(n.inv > 0.0f));  // (an infinite root, or no number)
  bool big = mine;
  if constexpr (TPR < 128 && TPR > 32) {
    if (tid == 0) overflow[local] = mine;
    __syncthreads();
    big = false;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) big |= overflow[i] != 0;
  }
  if (big) {
    const float f = tiny ? 0x1p80f : 0x1p-80f;
    const float ss2 = square_sum(f, false);
    if (mine) {
      n = inverse_rms(ss2, a, a.eps * f * f);
      const float back = tiny ? 0x1p80f : 0x1p-72f;
      n = Norm{tiny ? 1.0f : 0x1p-8f, n.inv * back, n.inv_lo * back};
    }
  }
  return n;
}

// v rounded to T: stored at p where there is one, and back in v.
__device__ __forceinline__ void round_store8(float* p, float (&v)[kVec]) {
  if (p) store8(p, v);
}
__device__ __forceinline__ void round_store8(bf16* p, float (&v)[kVec]) {
  Raw<bf16> r;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r.a);
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
  if (p) *reinterpret_cast<uint4*>(p) = r.a;
  values(r, v);
}

// Vector `at` of a row from its s in y (not `on`: past the row): y and its codes, as asked for.
template <typename T>
__device__ __forceinline__ void finish_vector(const NormArgs& a, int64_t row, int at, bool on, const Norm& n,
                                              const Raw<T>& rw, float (&y)[kVec]) {
  if (on) {
    if (n.scale != 1.0f) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) y[j] *= n.scale;
    }
    float lo[kVec];  // what the product's rounding and inv leave out
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float t = y[j] * n.inv;
      lo[j] = fmaf(y[j], n.inv_lo, fmaf(y[j], n.inv, -t));
      y[j] = t;
    }
    if (a.w) {
      float q[kVec];
      values(rw, q);
#pragma unroll
      for (int j = 0; j < kVec; ++j) y[j] = fmaf(y[j], q[j], lo[j] * q[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) y[j] += lo[j];
    }
    round_store8(a.y ? static_cast<T*>(a.y) + row * a.y_stride + at * kVec : nullptr, y);
  }
  if (!a.codes) return;
  float m = 0.0f;  // with codes, `on` is uniform over each 16 lanes (cols % 128 == 0)
  if (on) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) m = fmaxf(m, fabsf(y[j]));
  }
#pragma unroll
  for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (!on) return;
  const int e = ue8m0_exponent(m);
  const float sc = pow2_neg(e);
  reinterpret_cast<uint2*>(a.codes + row * a.cols)[at] =
      make_uint2(e4m3x4(y[0], y[1], y[2], y[3], sc), e4m3x4(y[4], y[5], y[6], y[7], sc));
  if ((at & 15) == 0) a.scale_bytes[row * (a.cols / 128) + (at >> 4)] = (uint8_t)(e + 127);
}

// ---- a row per block turn ----------------------------------------------------------
// Blocks an SM must hold, which bounds the registers: 768 threads (85 registers) for bf16 and 512 for
// binary32 (128; without the bound the compiler took 138, and 16384 x 7168 went from 301 to 370 us).
// Rows of a warp or two are quicker with more: bf16 with the 128 that let an SM hold four blocks (20000 x 1024 with a
// residual: 31 us; 36 with the 148 that the compiler would take), binary32 with as many as the compiler likes.
template <typename T, int TPR>
constexpr int kMinBlocks = TPR < 128 ? (sizeof(T) == 2 ? 4 : 1) : TPR > 256 ? 1 : (sizeof(T) == 2 ? 768 : 512) / TPR;

template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, kMinBlocks<T, TPR>) add_rmsnorm_kernel(NormArgs a) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  __shared__ float part[kRows][TPR > 32 ? TPR / 32 : 1];
  __shared__ int overflow[kRows];
  const int local = threadIdx.x / TPR, tid = threadIdx.x % TPR;
  const int vecs = a.cols / kVec;
  const int64_t blocks = (a.rows + kRows - 1) / kRows;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {  // every thread of the block takes every turn
    const int64_t row = b * kRows + local;
    const bool live = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.res_stride : nullptr;
    Raw<T> rx[NV], rr[NV], rw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * TPR + tid;
      if (live && at < vecs) {
        load8(rx[i], x + at * kVec);
        if (r) load8(rr[i], r + at * kVec);
        if (a.w) load8_weight(rw[i], static_cast<const T*>(a.w) + at * kVec);
      }
    }
    auto sum_of = [&](int i, float (&s)[kVec]) {  // s = x + r of vector i
      values(rx[i], s);
      if (!r) return;
      float q[kVec];
      values(rr[i], q);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[j] += q[j];
    };
    auto square_sum = [&](float scale, bool store) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = i * TPR + tid;
        if (!live || at >= vecs) continue;
        float s[kVec];
        sum_of(i, s);
        if (store && a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_stride + at * kVec, s);
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) t = fmaf(s[j] * scale, s[j] * scale, t);
        ss += t;
      }
      return row_sum<TPR>(ss, part[local]);
    };
    const Norm n = norm_of<TPR, kRows>(a, live, local, tid, overflow, square_sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * TPR + tid;
      const bool on = live && at < vecs;
      float y[kVec];
      if (on) sum_of(i, y);
      finish_vector<T>(a, row, at, on, n, rw[i], y);
    }
  }
}

// ---- many long rows ----------------------------------------------------------------
// Persistent blocks that keep the next rows' copies in flight (cp.async into slots of the thread
// that reads them: no barrier guards a slot), with the weight in registers.

__device__ __forceinline__ void copy16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(global)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

template <int TPR, int NV, int DEPTH, bool X_ONLY>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) add_rmsnorm_stream_kernel(NormArgs a) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  using T = bf16;
  extern __shared__ __align__(16) uint4 slots[];  // [DEPTH][x, r where there is one][NV][kThreads]
  __shared__ float part[kRows][TPR > 32 ? TPR / 32 : 1];
  __shared__ int overflow[kRows];
  const int local = threadIdx.x / TPR, tid = threadIdx.x % TPR;
  const int vecs = a.cols / kVec;
  const bool res = !X_ONLY && a.residual != nullptr;
  const int64_t blocks = (a.rows + kRows - 1) / kRows;
  Raw<T> rw[NV];
  if (a.w) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (i * TPR + tid < vecs) load8_weight(rw[i], static_cast<const T*>(a.w) + (i * TPR + tid) * kVec);
  }
  auto slot = [&](int d, int src, int i) { return slots + ((d * (1 + res) + src) * NV + i) * kThreads + threadIdx.x; };
  auto fetch = [&](int64_t b, int d) {
    const int64_t row = b * kRows + local;
    if (b < blocks && row < a.rows) {
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      const T* r = static_cast<const T*>(a.residual) + row * a.res_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = i * TPR + tid;
        if (at >= vecs) continue;
        copy16(slot(d, 0, i), x + at * kVec);
        if (res) copy16(slot(d, 1, i), r + at * kVec);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(blockIdx.x + (int64_t)d * gridDim.x, d);
  int d = 0;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {  // every thread of the block takes every turn
    const int64_t row = b * kRows + local;
    const bool live = row < a.rows;
    copies_wait<DEPTH - 1>();
    auto sum_of = [&](int i, float (&s)[kVec]) {  // s = x + r of vector i
      Raw<T> q;
      q.a = *slot(d, 0, i);
      values(q, s);
      if (!res) return;
      float t[kVec];
      q.a = *slot(d, 1, i);
      values(q, t);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[j] += t[j];
    };
    auto square_sum = [&](float scale, bool store) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = i * TPR + tid;
        if (!live || at >= vecs) continue;
        float s[kVec];
        sum_of(i, s);
        if (store && a.sum_out) store8(static_cast<T*>(a.sum_out) + row * a.sum_stride + at * kVec, s);
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) t = fmaf(s[j] * scale, s[j] * scale, t);
        ss += t;
      }
      return row_sum<TPR>(ss, part[local]);
    };
    const Norm n = norm_of<TPR, kRows>(a, live, local, tid, overflow, square_sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = i * TPR + tid;
      const bool on = live && at < vecs;
      float y[kVec];
      if (on) sum_of(i, y);
      finish_vector<T>(a, row, at, on, n, rw[i], y);
    }
    fetch(b + (int64_t)DEPTH * gridDim.x, d);  // this thread has read its slots
    if (++d == DEPTH) d = 0;
  }
}

template <typename T, int TPR, int NV>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  const int64_t blocks = ceil_div(a.rows, kRows);
  add_rmsnorm_kernel<T, TPR, NV><<<(unsigned)(blocks < (1 << 30) ? blocks : (1 << 30)), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int TPR, int NV, int DEPTH, bool X_ONLY>
cudaError_t launch_stream_t(const NormArgs& a, cudaStream_t s) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  constexpr size_t kSmem = (size_t)DEPTH * (X_ONLY ? 1 : 2) * NV * kThreads * 16;
  // blocks of an SM: by shared memory, and by registers (at most 85 a thread)
  constexpr int kFit = (int)(225000 / (kSmem + 1200)), kMost = kThreads >= 256 ? 768 / kThreads : 1536 / kThreads;
  constexpr int kPerSm = kFit < kMost ? kFit : kMost;
  static_assert(kPerSm >= 1, "shared memory");
  static std::atomic<uint64_t> attr;
  const cudaError_t e = set_smem_limit(attr, (const void*)add_rmsnorm_stream_kernel<TPR, NV, DEPTH, X_ONLY>, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = ceil_div(a.rows, kRows);
  add_rmsnorm_stream_kernel<TPR, NV, DEPTH, X_ONLY>
      <<<(unsigned)(blocks < 148 * kPerSm ? blocks : 148 * kPerSm), kThreads, kSmem, s>>>(a);
  return cudaGetLastError();
}

template <int TPR, int NV, int DEPTH>
cudaError_t launch_stream(const NormArgs& a, cudaStream_t s) {
  return a.residual ? launch_stream_t<TPR, NV, DEPTH, false>(a, s) : launch_stream_t<TPR, NV, DEPTH, true>(a, s);
}

// Few rows: a vector per thread, so that a row's latency is short. Many: four vectors per thread; for
// bf16 rows of up to 256 or over 4096 elements the streaming form (16384 x 7168 with residual, y and
// codes: 175 us against 207; 65536 x 256: 27 us against 33; but 4096 x 4096: 26.8 us against 23.1, and
// binary32 16384 x 7168: 389 us against 298).
template <typename T>
cudaError_t launch_t(const NormArgs& a, cudaStream_t s) {
  const int vecs = a.cols / kVec;
  if (a.rows <= kFewRows) {
    if (vecs <= 32) return launch_rows<T, 32, 1>(a, s);
    if (vecs <= 64) return launch_rows<T, 64, 1>(a, s);
    if (vecs <= 128) return launch_rows<T, 128, 1>(a, s);
    if (vecs <= 256) return launch_rows<T, 256, 1>(a, s);
    if (vecs <= 512) return launch_rows<T, 512, 1>(a, s);
    if (vecs <= 1024) return launch_rows<T, 1024, 1>(a, s);
    return launch_rows<T, 1024, 4>(a, s);
  }
  if constexpr (sizeof(T) == 2) {
    if (vecs <= 32) return launch_stream<32, 1, 3>(a, s);
    if (vecs > 512 && vecs <= 1024) return launch_stream<256, 4, 3>(a, s);
    if (vecs > 1024 && vecs <= 2048) return launch_stream<512, 4, 2>(a, s);
  }
  if (vecs <= 32) return launch_rows<T, 32, 1>(a, s);
  if (vecs <= 128) return launch_rows<T, 32, 4>(a, s);
  if (vecs <= 256) return launch_rows<T, 64, 4>(a, s);
  if (vecs <= 512) return launch_rows<T, 128, 4>(a, s);
  if (vecs <= 1024) return launch_rows<T, 256, 4>(a, s);
  if (vecs <= 2048) return launch_rows<T, 512, 4>(a, s);
  return launch_rows<T, 1024, 4>(a, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, int dtype, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.cols % kVec != 0 || a.cols > kNormMaxCols) return cudaErrorInvalidValue;
  return dtype == MOE_F32 ? launch_t<float>(a, s) : launch_t<bf16>(a, s);
}

}  // namespace moe
