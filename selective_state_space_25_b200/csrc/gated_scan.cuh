// gated_scan.cuh -- the gated linear recurrence: forward, backward, one-token
// step.
#pragma once

#include "block_common.cuh"

namespace ssm {

struct GatedParams {
  const void *u, *ga, *gx, *z;
  int64_t u_ld, ga_ld, gx_ld, z_ld;
  const float *A, *ba, *bx;
  const uint8_t *start;
  const float *h0;
  float *h_last;
  void *y;
  int64_t y_ld;
  float *chunk_h;
  int64_t b, L, d;
};

struct GatedBwdParams {
  GatedParams f;  // inputs of the forward; chunk_h is read
  const void *dout;
  int64_t dout_ld;
  const float *dh_last;
  void *du, *dga, *dgx, *dz;
  int64_t du_ld, dga_ld, dgx_ld, dz_ld;
  float *dh0;
  float *part;  // (parts, 3, d): sums of dA, dbias_a, dbias_x
};

struct GatedGate {
  float r, g, a, w;  // gates, decay, 1 - a^2
};

template <typename T>
__device__ __forceinline__ float act_load(const void *p, int64_t i, int64_t n) {
  return in_bounds(i, n, kBndAct) ? Elem<T>::load(static_cast<const T *>(p), i) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void act_store(void *p, int64_t i, int64_t n, float v) {
  if (in_bounds(i, n, kBndAct)) Elem<T>::store(static_cast<T *>(p), i, v);
}

__device__ __forceinline__ GatedGate gated_gate(float ga, float gx, float A2) {
  GatedGate o;
  o.r = sigmoid_f32(ga);
  o.g = sigmoid_f32(gx);
  float2 a, w;
  decay2(f2(A2 * o.r), a, w);
  o.a = a.x;
  o.w = w.x;
  return o;
}

// One thread per (batch, channel), the whole sequence in order.
template <typename T> __global__ void gated_fwd_kernel(const GatedParams p) {
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= p.b * p.d) return;
  const int64_t i = c / p.d, d = c % p.d, R = p.b * p.L;
  const float A2 = p.A[d] * kLog2e, ba = p.ba ? p.ba[d] : 0.0f, bx = p.bx ? p.bx[d] : 0.0f;
  float h = p.h0 ? p.h0[c] : 0.0f;
  const int64_t nC = (p.L + kGatedChunk - 1) / kGatedChunk;
  for (int64_t t = 0; t < p.L; ++t) {
    const int64_t r = i * p.L + t;
    if (p.chunk_h && t % kGatedChunk == 0) p.chunk_h[(i * nC + t / kGatedChunk) * p.d + d] = h;
    const float u = act_load<T>(p.u, r * p.u_ld + d, R * p.u_ld);
    const GatedGate q = gated_gate(act_load<T>(p.ga, r * p.ga_ld + d, R * p.ga_ld) + ba,
                                   act_load<T>(p.gx, r * p.gx_ld + d, R * p.gx_ld) + bx, A2);
    const float x = q.g * u;
    h = (p.start && p.start[r]) ? x : fmaf(q.a, h, sqrtf(q.w) * x);
    float y = h;
    if (p.z) y *= silu_f32(act_load<T>(p.z, r * p.z_ld + d, R * p.z_ld));
    act_store<T>(p.y, r * p.y_ld + d, R * p.y_ld, y);
  }
  if (p.h_last) p.h_last[c] = h;
}

// Backward in time, one thread per (batch, channel); a chunk's states are
// recomputed from its saved start state.
template <typename T> __global__ void gated_bwd_kernel(const GatedBwdParams q) {
  const GatedParams &p = q.f;
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= p.b * p.d) return;
  const int64_t i = c / p.d, d = c % p.d, R = p.b * p.L;
  const float A = p.A[d], A2 = A * kLog2e, ba = p.ba ? p.ba[d] : 0.0f, bx = p.bx ? p.bx[d] : 0.0f;
  const int64_t nC = (p.L + kGatedChunk - 1) / kGatedChunk;
  float mu = q.dh_last ? q.dh_last[c] : 0.0f;  // a_{t+1} lam_{t+1}
  float sA = 0.0f, sa = 0.0f, sx = 0.0f;
  float prev[kGatedChunk];
  for (int64_t k = nC - 1; k >= 0; --k) {
    const int64_t t0 = k * kGatedChunk;
    const int n = (int)(p.L - t0 < kGatedChunk ? p.L - t0 : kGatedChunk);
    float h = p.chunk_h[(i * nC + k) * p.d + d];
    for (int t = 0; t < n; ++t) {
      const int64_t r = i * p.L + t0 + t;
      prev[t] = h;
      const GatedGate g = gated_gate(act_load<T>(p.ga, r * p.ga_ld + d, R * p.ga_ld) + ba,
                                     act_load<T>(p.gx, r * p.gx_ld + d, R * p.gx_ld) + bx, A2);
      const float x = g.g * act_load<T>(p.u, r * p.u_ld + d, R * p.u_ld);
      h = (p.start && p.start[r]) ? x : fmaf(g.a, h, sqrtf(g.w) * x);
    }
    for (int t = n - 1; t >= 0; --t) {
      const int64_t r = i * p.L + t0 + t;
      const bool st = p.start && p.start[r];
      const GatedGate g = gated_gate(act_load<T>(p.ga, r * p.ga_ld + d, R * p.ga_ld) + ba,
                                     act_load<T>(p.gx, r * p.gx_ld + d, R * p.gx_ld) + bx, A2);
      const float u = act_load<T>(p.u, r * p.u_ld + d, R * p.u_ld);
      const float dout = act_load<T>(q.dout, r * q.dout_ld + d, R * q.dout_ld);
      const float f = st ? 1.0f : sqrtf(g.w);
      float go = dout;
      if (p.z) {
        const float z = act_load<T>(p.z, r * p.z_ld + d, R * p.z_ld);
        const float s = sigmoid_f32(z);
        const float ht = st ? g.g * u : fmaf(g.a, prev[t], f * g.g * u);
        go = dout * z * s;
        act_store<T>(q.dz, r * q.dz_ld + d, R * q.dz_ld, dout * ht * s * (1.0f + z * (1.0f - s)));
      }
      const float lam = go + mu;
      const float dl = st ? 0.0f
                          : lam * (g.a * prev[t] -
                                   (g.w > 0.0f ? g.a * g.a * g.g * u * rsqrt_approx(g.w) : 0.0f));
      const float dga = dl * A * g.r * (1.0f - g.r);
      const float dgx = lam * f * u * g.g * (1.0f - g.g);
      act_store<T>(q.du, r * q.du_ld + d, R * q.du_ld, lam * f * g.g);
      act_store<T>(q.dga, r * q.dga_ld + d, R * q.dga_ld, dga);
      act_store<T>(q.dgx, r * q.dgx_ld + d, R * q.dgx_ld, dgx);
      sA = fmaf(dl, g.r, sA);
      sa += dga;
      sx += dgx;
      mu = st ? 0.0f : g.a * lam;
    }
  }
  if (q.dh0) q.dh0[c] = mu;
  q.part[(i * 3 + 0) * p.d + d] = sA;
  q.part[(i * 3 + 1) * p.d + d] = sa;
  q.part[(i * 3 + 2) * p.d + d] = sx;
}

// One token, one thread per (row, channel): bound by the state's read and
// write and the activations.
template <typename T> __global__ void gated_step_kernel(const GatedParams p, float *state) {
  const int64_t c = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (c >= p.b * p.d) return;
  const int64_t i = c / p.d, d = c % p.d;
  const float A2 = p.A[d] * kLog2e, ba = p.ba ? p.ba[d] : 0.0f, bx = p.bx ? p.bx[d] : 0.0f;
  const GatedGate q = gated_gate(act_load<T>(p.ga, i * p.ga_ld + d, p.b * p.ga_ld) + ba,
                                 act_load<T>(p.gx, i * p.gx_ld + d, p.b * p.gx_ld) + bx, A2);
  const float h = fmaf(q.a, state[c], sqrtf(q.w) * (q.g * act_load<T>(p.u, i * p.u_ld + d, p.b * p.u_ld)));
  state[c] = h;
  float y = h;
  if (p.z) y *= silu_f32(act_load<T>(p.z, i * p.z_ld + d, p.b * p.z_ld));
  act_store<T>(p.y, i * p.y_ld + d, p.b * p.y_ld, y);
}

}  // namespace ssm
