// block_common.cuh -- device helpers shared by the kernels around the scan
// (gated recurrence, causal convolution, norms).
#pragma once

#include "ssm_common.cuh"

namespace ssm {

// Steps between the states that ssm_gated_scan_fwd keeps for its backward.
constexpr int kGatedChunk = 32;

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

// max that keeps a NaN operand.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }

// Decays of two elements from x = A r log2(e) <= 0: a = 2^x and w = 1 - a^2 +
// kDecayMinW, both with the accuracy the recurrence needs.  x = j + s with j =
// rint(x), S = 2^j: a = S + S p, a - 1 = S p + (S - 1) with p = 2^s - 1 the
// polynomial; for j = 0 that is p itself, below it S - 1 is exact and no smaller
// than 1/2.  w = -(a - 1)(a + 1); the 1e-36 keeps its inverse root finite where a
// is 1.  x > 0 (A > 0, outside the operator's domain) makes w negative and what
// its root enters NaN.
constexpr float kDecayMinW = 1e-36f;
__device__ __forceinline__ void decay2(float2 x, float2 &a, float2 &w) {
  x.x = max_nan(x.x, -126.0f);
  x.y = max_nan(x.y, -126.0f);
  const float2 t = __fadd2_rn(x, f2(12582912.0f));  // 1.5 2^23: the low bits hold rint(x)
  const float2 j = __fadd2_rn(t, f2(-12582912.0f));
  const float2 s = __ffma2_rn(j, f2(-1.0f), x);     // x - j, exact
  float2 q = __ffma2_rn(f2(kDecayQ5), s, f2(kDecayQ4));
  q = __ffma2_rn(q, s, f2(kDecayQ3));
  q = __ffma2_rn(q, s, f2(kDecayQ2));
  q = __ffma2_rn(q, s, f2(kDecayQ1));
  q = __ffma2_rn(q, s, f2(kDecayQ0));
  const float2 p = __fmul2_rn(q, s);
  const float2 S = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                               __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
  a = __ffma2_rn(S, p, S);
  const float2 m = __ffma2_rn(S, p, __fadd2_rn(S, f2(-1.0f)));
  w = __ffma2_rn(m, __ffma2_rn(m, f2(-1.0f), f2(-2.0f)), f2(kDecayMinW));
}

// ------------------------------------------------------- element access
// VEC adjacent elements of an activation as one access (VEC * sizeof(T) bytes,
// so aligned), in fp32 registers.  `n`: elements of the buffer up to the end of
// its last row, for the debug-bounds build.
template <typename T, int VEC> struct VecWord;
template <> struct VecWord<__nv_bfloat16, 1> { using type = uint16_t; };
template <> struct VecWord<__nv_bfloat16, 2> { using type = uint32_t; };
template <> struct VecWord<__nv_bfloat16, 4> { using type = uint2; };
template <> struct VecWord<__nv_bfloat16, 8> { using type = uint4; };
template <> struct VecWord<float, 1> { using type = float; };
template <> struct VecWord<float, 2> { using type = float2; };
template <> struct VecWord<float, 4> { using type = float4; };

// A load through the non-coherent path, for data no one writes meanwhile.
template <typename T, int VEC>
__device__ __forceinline__ typename VecWord<T, VEC>::type ld_raw_ro(const void *p, int64_t i,
                                                                    int64_t n) {
  using W = typename VecWord<T, VEC>::type;
  if (in_bounds(i, n - (VEC - 1), kBndAct))
    return __ldg(reinterpret_cast<const W *>(static_cast<const T *>(p) + i));
  return W{};
}
__device__ __forceinline__ void unpack(uint16_t w, float *v) { v[0] = bf16lo(w); }
__device__ __forceinline__ void unpack(uint32_t w, float *v) {
  v[0] = bf16lo(w);
  v[1] = bf16hi(w);
}
__device__ __forceinline__ void unpack(uint2 w, float *v) {
  unpack(w.x, v);
  unpack(w.y, v + 2);
}
__device__ __forceinline__ void unpack(uint4 w, float *v) {
  unpack(w.x, v);
  unpack(w.y, v + 2);
  unpack(w.z, v + 4);
  unpack(w.w, v + 6);
}
__device__ __forceinline__ void unpack(float w, float *v) { v[0] = w; }
__device__ __forceinline__ void unpack(float2 w, float *v) {
  v[0] = w.x;
  v[1] = w.y;
}
__device__ __forceinline__ void unpack(float4 w, float *v) {
  v[0] = w.x;
  v[1] = w.y;
  v[2] = w.z;
  v[3] = w.w;
}
// VEC values rounded once to T and stored as one access.
template <typename T, int VEC>
__device__ __forceinline__ void st_vec(void *p, int64_t i, int64_t n, const float *v) {
  using W = typename VecWord<T, VEC>::type;
  if (!in_bounds(i, n - (VEC - 1), kBndAct)) return;
  T *q = static_cast<T *>(p) + i;
  if constexpr (sizeof(T) == 4) {
    if constexpr (VEC == 1) *q = v[0];
    if constexpr (VEC == 2) *reinterpret_cast<W *>(q) = make_float2(v[0], v[1]);
    if constexpr (VEC == 4) *reinterpret_cast<W *>(q) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    if constexpr (VEC == 1) *q = __float2bfloat16_rn(v[0]);
    if constexpr (VEC == 2) *reinterpret_cast<W *>(q) = pack_bf16x2(v[0], v[1]);
    if constexpr (VEC == 4)
      *reinterpret_cast<W *>(q) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    if constexpr (VEC == 8)
      *reinterpret_cast<W *>(q) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}
// Arithmetic on one value or a packed pair (two to an instruction: the same rate a
// lane, half the issue slots).
__device__ __forceinline__ float mulv(float a, float b) { return a * b; }
__device__ __forceinline__ float addv(float a, float b) { return a + b; }
__device__ __forceinline__ float fmav(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 mulv(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 addv(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fmav(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mulv(float2 a, float b) { return __fmul2_rn(a, f2(b)); }
__device__ __forceinline__ float ex2v(float x) { return ex2_approx(x); }
__device__ __forceinline__ float2 ex2v(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float rcpv(float x) { return rcp_approx(x); }
__device__ __forceinline__ float2 rcpv(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
template <typename F> __device__ __forceinline__ F bc(float v);
template <> __device__ __forceinline__ float bc<float>(float v) { return v; }
template <> __device__ __forceinline__ float2 bc<float2>(float v) { return f2(v); }
__device__ __forceinline__ float hsum(float v) { return v; }
__device__ __forceinline__ float hsum(float2 v) { return v.x + v.y; }
template <typename F> __device__ __forceinline__ F sigmoidv(F x) {
  return rcpv(addv(ex2v(mulv(x, bc<F>(-kLog2e))), bc<F>(1.0f)));
}
// E values as pairs where E allows.
template <int E> struct Lanes {
  using F = float2;
  static constexpr int N = E / 2;
};
template <> struct Lanes<1> {
  using F = float;
  static constexpr int N = 1;
};

// acc += a * b over VEC values, two to an instruction (packed fp32: the same
// rate a lane, half the issue slots).
template <int VEC>
__device__ __forceinline__ void fma_vec(float *acc, const float *a, const float *b) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 r = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]),
                                  make_float2(acc[e], acc[e + 1]));
      acc[e] = r.x;
      acc[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = fmaf(a[e], b[e], acc[e]);
  }
}

__device__ __forceinline__ float ld_param(const float *p, int64_t i, int64_t n) {
  return in_bounds(i, n, kBndParam) ? __ldg(p + i) : 0.0f;
}

// Elements from a buffer's first to the end of its last row.
__device__ __forceinline__ int64_t extent(int64_t rows, int64_t d, int64_t ld) {
  return (rows - 1) * ld + d;
}

__device__ __forceinline__ float sigmoid_f32(float x) {
  return rcp_approx(1.0f + ex2_approx(-x * kLog2e));
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
  grid_dependency_wait();
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
