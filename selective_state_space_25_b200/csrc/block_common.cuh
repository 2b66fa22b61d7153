// block_common.cuh -- device helpers shared by the kernels around the scan
// (gated recurrence, causal convolution, norms).
#pragma once

#include "ssm_common.cuh"

namespace ssm {

// Steps between the states ssm_gated_scan_fwd keeps for its backward.
constexpr int kGatedChunk = 64;

// Largest convolution width.
constexpr int kMaxConv = 8;

// 2^(x) - 1 on [-1/2, 1/2] as x q(x), q of degree 5: the minimax fit of
// fit_polys.py (fit_exp2(5)), relative error 2.2e-8.  The recurrence needs
// 1 - a for decays near 1 to full relative accuracy: the state's memory is
// 1 / (1 - a) steps long and the input factor is sqrt(1 - a^2).
constexpr float kDecayQ0 = 6.931471825e-01f;
constexpr float kDecayQ1 = 2.402264923e-01f;
constexpr float kDecayQ2 = 5.550357327e-02f;
constexpr float kDecayQ3 = 9.618237615e-03f;
constexpr float kDecayQ4 = 1.339073526e-03f;
constexpr float kDecayQ5 = 1.540351223e-04f;

// max / min that keep a NaN operand.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }

// Decays of two elements from x = A r log2(e): a = 2^x and w = 1 - a^2, both
// with the accuracy the recurrence needs.  x = j + s with j = rint(x); for
// j = 0 a - 1 is the polynomial itself, below it a <= 2^-1/2 and a - 1 loses
// nothing.  w = -(a - 1)(a + 1), at least 0.
__device__ __forceinline__ void decay2(float2 x, float2 &a, float2 &w) {
  x.x = min_nan(max_nan(x.x, -126.0f), 126.0f);
  x.y = min_nan(max_nan(x.y, -126.0f), 126.0f);
  const float2 t = __fadd2_rn(x, f2(12582912.0f));  // 1.5 2^23: the low bits hold rint(x)
  const float2 j = __fadd2_rn(t, f2(-12582912.0f));
  const float2 s = __ffma2_rn(j, f2(-1.0f), x);     // x - j, exact
  float2 q = __ffma2_rn(f2(kDecayQ5), s, f2(kDecayQ4));
  q = __ffma2_rn(q, s, f2(kDecayQ3));
  q = __ffma2_rn(q, s, f2(kDecayQ2));
  q = __ffma2_rn(q, s, f2(kDecayQ1));
  q = __ffma2_rn(q, s, f2(kDecayQ0));
  float2 m = __fmul2_rn(q, s);
  a = __fadd2_rn(m, f2(1.0f));
  a.x = __int_as_float(__float_as_int(a.x) + (__float_as_int(t.x) << 23));
  a.y = __int_as_float(__float_as_int(a.y) + (__float_as_int(t.y) << 23));
  const float2 m1 = __fadd2_rn(a, f2(-1.0f));
  m.x = j.x == 0.0f ? m.x : m1.x;
  m.y = j.y == 0.0f ? m.y : m1.y;
  // -m (2 + m)
  const float2 n = __ffma2_rn(m, f2(-1.0f), f2(-2.0f));
  w = __fmul2_rn(m, n);
  w.x = max_nan(w.x, 0.0f);
  w.y = max_nan(w.y, 0.0f);
}

// Sums of partial rows, the last step of the parameters' gradients: column c
// of the m0 + m1 + m2 columns is sum_n part[n, c], taken by eight lanes in
// order of n and then over the lanes (the same bits every time); it goes to
// out0, out1 or out2, where the call wants it.
constexpr int kColSumCols = 32, kColSumRows = 8;
struct ColSumParams {
  const float *part;
  int64_t n, m0, m1, m2;
  float *out0, *out1, *out2;
};
__global__ void col_sum_kernel(const ColSumParams p) {
  __shared__ float s[kColSumRows][kColSumCols + 1];
  const int64_t m = p.m0 + p.m1 + p.m2;
  const int64_t c = blockIdx.x * (int64_t)kColSumCols + threadIdx.x;
  float acc = 0.0f;
  if (c < m) {
#pragma unroll 4
    for (int64_t i = threadIdx.y; i < p.n; i += kColSumRows)
      if (in_bounds(i * m + c, p.n * m, kBndWork)) acc += p.part[i * m + c];
  }
  s[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.y != 0 || c >= m) return;
#pragma unroll
  for (int k = 1; k < kColSumRows; ++k) acc += s[k][threadIdx.x];
  float *out = c < p.m0 ? p.out0 : c < p.m0 + p.m1 ? p.out1 : p.out2;
  const int64_t o = c < p.m0 ? c : c < p.m0 + p.m1 ? c - p.m0 : c - p.m0 - p.m1;
  const int64_t no = c < p.m0 ? p.m0 : c < p.m0 + p.m1 ? p.m1 : p.m2;
  if (out && in_bounds(o, no, kBndParam)) out[o] = acc;
}

}  // namespace ssm
