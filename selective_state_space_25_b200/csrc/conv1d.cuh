// conv1d.cuh -- the causal depthwise convolution over a sequence: forward,
// backward, one-token step.
#pragma once

#include "block_common.cuh"
#include "gated_scan.cuh"

namespace ssm {

struct ConvParams {
  const void *x;
  int64_t x_ld;
  const float *w, *bias;
  int silu;
  const void *win;   // window in front of the sequence, nullable
  void *win_out;     // window behind it, nullable
  const uint8_t *start;
  void *y;
  int64_t y_ld;
  int64_t b, L, d;
  int K;
};

struct ConvBwdParams {
  ConvParams f;
  const void *dy;
  int64_t dy_ld;
  void *dx;
  int64_t dx_ld;
  float *part;  // (parts, d (K + 1)): sums of dweight, then dbias
};

// Input of step t of sequence i (t < 0: the window's entry, or 0).
template <typename T>
__device__ __forceinline__ float conv_in(const ConvParams &p, int64_t i, int64_t t, int64_t d) {
  if (t >= 0) {
    const int64_t r = i * p.L + t;
    return act_load<T>(p.x, r * p.x_ld + d, p.b * p.L * p.x_ld);
  }
  if (!p.win) return 0.0f;
  return act_load<T>(p.win, (i * p.d + d) * p.K + p.K + t, p.b * p.d * p.K);
}

// One thread per (batch, channel): the window slides over the sequence in
// registers.
template <typename T> __global__ void conv_fwd_kernel(const ConvParams p) {
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= p.b * p.d) return;
  const int64_t i = c / p.d, d = c % p.d;
  float w[kMaxConv], v[kMaxConv];
  for (int j = 0; j < p.K; ++j) {
    w[j] = p.w[d * p.K + j];
    v[j] = conv_in<T>(p, i, j - p.K, d);
  }
  const float bias = p.bias ? p.bias[d] : 0.0f;
  for (int64_t t = 0; t < p.L; ++t) {
    const bool st = p.start && p.start[i * p.L + t];
    for (int j = 0; j + 1 < p.K; ++j) v[j] = st ? 0.0f : v[j + 1];
    v[p.K - 1] = conv_in<T>(p, i, t, d);
    float s = bias;
    for (int j = 0; j < p.K; ++j) s = fmaf(w[j], v[j], s);
    const int64_t r = i * p.L + t;
    act_store<T>(p.y, r * p.y_ld + d, p.b * p.L * p.y_ld, p.silu ? silu_f32(s) : s);
  }
  if (p.win_out)
    for (int j = 0; j < p.K; ++j) act_store<T>(p.win_out, c * p.K + j, p.b * p.d * p.K, v[j]);
}

template <typename T> __global__ void conv_bwd_kernel(const ConvBwdParams q) {
  const ConvParams &p = q.f;
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= p.b * p.d) return;
  const int64_t i = c / p.d, d = c % p.d, R = p.b * p.L;
  const int K = p.K;
  float w[kMaxConv], v[kMaxConv], g[kMaxConv], dw[kMaxConv];  // g[m]: dx of step t - m so far
  for (int j = 0; j < K; ++j) {
    w[j] = p.w[d * K + j];
    v[j] = conv_in<T>(p, i, j - K, d);
    dw[j] = g[j] = 0.0f;
  }
  const float bias = p.bias ? p.bias[d] : 0.0f;
  float db = 0.0f;
  int64_t first = -(int64_t)K;  // the current sequence's first step
  for (int64_t t = 0; t < p.L; ++t) {
    const int64_t r = i * p.L + t;
    const bool st = p.start && p.start[r];
    if (st) first = t;
    for (int j = 0; j + 1 < K; ++j) v[j] = st ? 0.0f : v[j + 1];
    v[K - 1] = conv_in<T>(p, i, t, d);
    float s = bias;
    for (int j = 0; j < K; ++j) s = fmaf(w[j], v[j], s);
    float dp = act_load<T>(q.dy, r * q.dy_ld + d, R * q.dy_ld);
    if (p.silu) {
      const float sg = sigmoid_f32(s);
      dp *= sg * (1.0f + s * (1.0f - sg));
    }
    db += dp;
    for (int m = K - 1; m > 0; --m) g[m] = g[m - 1];
    g[0] = 0.0f;
    for (int m = 0; m < K; ++m)
      if (t - m >= first) {  // taps before the sequence's start take no gradient
        g[m] = fmaf(w[K - 1 - m], dp, g[m]);
        dw[K - 1 - m] = fmaf(v[K - 1 - m], dp, dw[K - 1 - m]);
      }
    if (t - K + 1 >= 0)
      act_store<T>(q.dx, (r - K + 1) * q.dx_ld + d, R * q.dx_ld, g[K - 1]);
  }
  for (int m = K - 2; m >= 0; --m)  // the last K - 1 steps
    if (p.L - 1 - m >= 0)
      act_store<T>(q.dx, (i * p.L + p.L - 1 - m) * q.dx_ld + d, R * q.dx_ld, g[m]);
  float *part = q.part + i * p.d * (K + 1);
  for (int j = 0; j < K; ++j) part[d * K + j] = dw[j];
  part[p.d * K + d] = db;
}

template <typename T> __global__ void conv_step_kernel(const ConvParams p, void *win) {
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= p.b * p.d) return;
  const int64_t i = c / p.d, d = c % p.d, n = p.b * p.d * p.K;
  float s = p.bias ? p.bias[d] : 0.0f;
  for (int j = 0; j < p.K; ++j) {
    const float v = j + 1 < p.K ? act_load<T>(win, c * p.K + j + 1, n)
                                : act_load<T>(p.x, i * p.x_ld + d, p.b * p.x_ld);
    act_store<T>(win, c * p.K + j, n, v);
    s = fmaf(p.w[d * p.K + j], v, s);
  }
  act_store<T>(p.y, i * p.y_ld + d, p.b * p.y_ld, p.silu ? silu_f32(s) : s);
}

}  // namespace ssm
