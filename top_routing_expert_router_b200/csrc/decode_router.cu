// decode_router.cu -- first kernel of the layers for few tokens: the router logits in binary64, the
// E4M3 tiles of x for FP8 experts, and cleared counters (decode.cuh has the scheme).
//
//   logit[t, e] = x_t . W_r[e]
// Reads W_r once per 16 tokens and x once per pair of experts; at one token it is bound by latency
// (one round of loads), at 64 by the binary64 products (117 million at E = 256, d = 7168).
#include <limits.h>

#include "decode.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kChunkTokens = 16;  // tokens of a block

// The codes of a 1 x 128 tile, four values per lane of the warp, and its scale byte.
__device__ __forceinline__ uint32_t quantize_tile(const float (&v)[4], uint32_t* byte) {
  float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  const int e = ue8m0_exponent(m);
  *byte = (uint32_t)(e + 127);
  return e4m3x4(v[0], v[1], v[2], v[3], pow2_neg(e));
}

// Tile i of x's n * d / 128 (row by row), by one warp.
__device__ __forceinline__ void quantize_x_tile(const DecodeArgs& a, int64_t i) {
  const int lane = threadIdx.x & 31;
  const uint2 raw = __ldg(reinterpret_cast<const uint2*>(a.x) + i * 32 + lane);
  const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u), __uint_as_float(raw.y << 16),
                      __uint_as_float(raw.y & 0xFFFF0000u)};
  uint32_t byte;
  const uint32_t q = quantize_tile(v, &byte);
  reinterpret_cast<uint32_t*>(a.xq)[i * 32 + lane] = q;
  if (lane == 0) a.xs[i] = (uint8_t)byte;
}

// 16 bytes of activations or router weights as binary32 (8 bf16 or 4 binary32 values).
template <typename T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);
};
__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[8]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[4]) {
  v[0] = __uint_as_float(raw.x), v[1] = __uint_as_float(raw.y), v[2] = __uint_as_float(raw.z), v[3] = __uint_as_float(raw.w);
}

// A binary32 value times 2^-896 as a binary64, exact for every finite value (subnormals and zeros
// included: the fields only move): three integer operations, where the conversion instruction runs
// at 4 lanes a clock and SM and made the logits of 64 tokens take 150 us.
__device__ __forceinline__ double widened(float v) {
  const int u = __float_as_int(v);
  return __hiloint2double((u >> 3) & (int)0x8FFFFFFF, u << 29);
}
// A router weight gets 2^512 (two steps: 2^(896 + 512) is past the range), so that its products with
// widened activations are 2^-384 of the true ones, far from both ends of the range.
__device__ __forceinline__ double widened_weight(float v) { return widened(v) * 0x1p1000 * 0x1p408; }
constexpr double kWidenLogit = 0x1p384;

constexpr int kRouterTokens = 4;  // tokens of one dot-product item: each weight is widened once for them

// Binary64 logits of experts e0 and (pair) e0 + 1 for tokens [first, end), by the NW warps of a block
// (`part`: NW * 2 * TOK doubles). Products of bf16 values are exact, sums are binary64. Items are groups of TOK tokens, cut along d when there are fewer of them than warps; a cut item's
// parts are added in order. The loads of BATCH steps are issued before their products: a step whose
// loads wait on branches took a memory latency per token. A row with a NaN or an infinity gets NaN
// logits (the widening alone would take them for finite values).
template <typename T, int NW, int TOK, int BATCH>
__device__ void logits_pair(const DecodeArgs& a, int e0, bool pair, int first, int end, double* part) {
  constexpr int C = Chunk<T>::N;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int items = (end - first + TOK - 1) / TOK;
  const int cuts = items >= NW ? 1 : NW / items;
  const int chunks = a.d / C;  // d % 8 == 0
  const int per = (chunks + cuts - 1) / cuts;
  const uint4* w0 = reinterpret_cast<const uint4*>(static_cast<const T*>(a.w_router) + (int64_t)e0 * a.d);
  const uint4* w1 = pair ? w0 + chunks : w0;
  for (int it = w; it < items * cuts; it += NW) {
    const int item = it / cuts, cut = it % cuts, t0 = first + item * TOK;
    const int last = min(TOK, end - t0) - 1;
    const uint4* xr = reinterpret_cast<const uint4*>(a.x) + (int64_t)t0 * chunks;
    double acc[2][TOK] = {};
    float odd[2] = {}, odd_x[TOK] = {};  // NaN once a value is not finite
    const int c1 = min(chunks, (cut + 1) * per);
    for (int c0 = cut * per; c0 < c1; c0 += 32 * BATCH) {
      uint4 r0[BATCH], r1[BATCH], rx[BATCH][TOK];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int c = c0 + 32 * b + lane;
        const bool in = c < c1;
        r0[b] = in ? __ldg(w0 + c) : make_uint4(0, 0, 0, 0);
        r1[b] = in ? __ldg(w1 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < TOK; ++q)  // past the last token: its row again, not stored
          rx[b][q] = in ? __ldg(xr + (int64_t)min(q, last) * chunks + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        float v0[C], v1[C];
        unpack(r0[b], v0);
        unpack(r1[b], v1);
        double d0[C], d1[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
          d0[j] = widened_weight(v0[j]);
          d1[j] = widened_weight(v1[j]);
          odd[0] = fmaf(v0[j], 0.0f, odd[0]);
          odd[1] = fmaf(v1[j], 0.0f, odd[1]);
        }
#pragma unroll
        for (int q = 0; q < TOK; ++q) {
          float xv[C];
          unpack(rx[b][q], xv);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const double xd = widened(xv[j]);
            acc[0][q] = fma(xd, d0[j], acc[0][q]);
            acc[1][q] = fma(xd, d1[j], acc[1][q]);
            odd_x[q] = fmaf(xv[j], 0.0f, odd_x[q]);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < TOK; ++q)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const double s = warp_sum(acc[p][q] * kWidenLogit + (double)(odd[p] + odd_x[q]));
        if (lane != 0 || (p && !pair) || q > last) continue;
        if (cuts == 1)
          a.logits[(int64_t)(t0 + q) * a.E + e0 + p] = s;
        else
          part[(it * 2 + p) * TOK + q] = s;  // it < items * cuts <= NW
      }
  }
  if (cuts == 1) return;
  __syncthreads();
  if (w == 0)
    for (int i = lane; i < items * 2 * TOK; i += 32) {
      const int item = i / (2 * TOK), p = i / TOK % 2, q = i % TOK;
      const int t = first + item * TOK + q;
      if (t >= end || (p && !pair)) continue;
      double s = 0.0;
      for (int cut = 0; cut < cuts; ++cut) s += part[((item * cuts + cut) * 2 + p) * TOK + q];
      a.logits[(int64_t)t * a.E + e0 + p] = s;
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) decode_router_kernel(DecodeArgs a, int quants, int pairs) {
  __shared__ double part[kWarps * 2 * kRouterTokens];
  wait_for_earlier_kernels();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the layer's kernel sets itself up meanwhile
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.ctr_bytes / 16; i += 32 * kWarps) reinterpret_cast<uint4*>(a.ctr)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) a.status->status = MOE_OK;
    if (a.test_stall) {  // counts that never reach what is waited for
      __syncthreads();
      if (a.test_stall == 1)
        for (int e = threadIdx.x; e <= a.E; e += 32 * kWarps) a.ctr[kCtrExpert + e] = INT_MIN;
      else if (threadIdx.x == 0)
        a.ctr[kCtrTokenDone] = INT_MIN;
    }
  }
  const int u = blockIdx.x;
  if (u < quants) {
    const int i = u * kWarps + (threadIdx.x >> 5);
    if (i < a.n * (a.d / 128)) quantize_x_tile(a, i);
    return;
  }
  const int e0 = (u - quants) % pairs * 2, first = (u - quants) / pairs * kChunkTokens;
  const int end = min(a.n, first + kChunkTokens);
  if (a.n == 1)
    logits_pair<T, kWarps, 1, 4>(a, e0, e0 + 1 < a.E, first, end, part);
  else
    logits_pair<T, kWarps, kRouterTokens, 2>(a, e0, e0 + 1 < a.E, first, end, part);
}

}  // namespace

cudaError_t launch_decode_router(const DecodeArgs& a, cudaStream_t s) {
  const int quants = a.quantize ? (int)ceil_div((int64_t)a.n * (a.d / 128), kWarps) : 0;
  const int pairs = (a.E + 1) / 2, grid = quants + pairs * (int)ceil_div(a.n, kChunkTokens);
  if (a.dtype == MOE_F32) return launch_early(decode_router_kernel<float>, grid, 32 * kWarps, 0, s, a, quants, pairs);
  return launch_early(decode_router_kernel<bf16>, grid, 32 * kWarps, 0, s, a, quants, pairs);
}

}  // namespace moe
