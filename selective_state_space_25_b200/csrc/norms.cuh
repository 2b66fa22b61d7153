// norms.cuh -- the gated RMS norm and the residual-add norm, forward and
// backward.
#pragma once

#include "block_common.cuh"

namespace ssm {

template <typename T>
__device__ __forceinline__ float act_load(const void *p, int64_t i, int64_t n) {
  return in_bounds(i, n, kBndAct) ? Elem<T>::load(static_cast<const T *>(p), i) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void act_store(void *p, int64_t i, int64_t n, float v) {
  if (in_bounds(i, n, kBndAct)) Elem<T>::store(static_cast<T *>(p), i, v);
}

struct GatedNormParams {
  const void *x, *z;
  int64_t x_ld, z_ld;
  const float *w;
  int64_t groups;
  float eps;
  int before;  // norm before gate
  void *y;
  int64_t y_ld;
  int64_t rows, d;
};
struct GatedNormBwdParams {
  GatedNormParams f;
  const void *dy;
  int64_t dy_ld;
  void *dx, *dz;
  int64_t dx_ld, dz_ld;
  float *part;  // (parts, d)
};
struct AddNormParams {
  const void *x, *res;
  int64_t x_ld, res_ld;
  const float *w, *post, *scale;
  float eps;
  void *y, *res_out;
  int64_t y_ld, ro_ld;
  int64_t rows, d;
};
struct AddNormBwdParams {
  AddNormParams f;  // res_out is read
  const void *dy, *dro;
  int64_t dy_ld, dro_ld;
  void *dx, *dres;
  int64_t dx_ld, dres_ld;
  float *part;  // (parts, 3, d): dweight, dpost_weight, dscale
};

constexpr int kNormThreads = 256;

// Sum over the CTA, the same value in every thread.
__device__ __forceinline__ float cta_sum(float v, float *s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
  for (int k = 0; k < kNormThreads / 32; ++k) v += s[k];
  return v;
}

template <typename T> __global__ void gated_norm_fwd_kernel(const GatedNormParams p) {
  __shared__ float s[32];
  const int64_t n = p.d / p.groups;
  for (int64_t k = blockIdx.x; k < p.rows * p.groups; k += gridDim.x) {
    const int64_t r = k / p.groups, c0 = k % p.groups * n;
    float ss = 0.0f;
    for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
      float v = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld);
      if (p.z && !p.before) v *= silu_f32(act_load<T>(p.z, r * p.z_ld + c, p.rows * p.z_ld));
      ss = fmaf(v, v, ss);
    }
    const float rs = rsqrtf(cta_sum(ss, s) / (float)n + p.eps);
    for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
      float v = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld) * rs * p.w[c];
      if (p.z) v *= silu_f32(act_load<T>(p.z, r * p.z_ld + c, p.rows * p.z_ld));
      act_store<T>(p.y, r * p.y_ld + c, p.rows * p.y_ld, v);
    }
  }
}

template <typename T> __global__ void gated_norm_bwd_kernel(const GatedNormBwdParams q) {
  __shared__ float s[32];
  const GatedNormParams &p = q.f;
  const int64_t n = p.d / p.groups;
  float *part = q.part + blockIdx.x * p.d;
  for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) part[c] = 0.0f;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x)
    for (int64_t c0 = 0; c0 < p.d; c0 += n) {
      __syncthreads();
      float ss = 0.0f, sd = 0.0f;
      for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld);
        const float gate = p.z ? silu_f32(act_load<T>(p.z, r * p.z_ld + c, p.rows * p.z_ld)) : 1.0f;
        const float dy = act_load<T>(q.dy, r * q.dy_ld + c, p.rows * q.dy_ld);
        const float v = p.before ? x : x * gate, dn = dy * p.w[c] * (p.before ? gate : 1.0f);
        ss = fmaf(v, v, ss);
        sd = fmaf(dn, v, sd);
      }
      const float rs = rsqrtf(cta_sum(ss, s) / (float)n + p.eps);
      const float k = cta_sum(sd, s) * rs * rs / (float)n;
      for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld);
        const float z = p.z ? act_load<T>(p.z, r * p.z_ld + c, p.rows * p.z_ld) : 0.0f;
        const float sg = sigmoid_f32(z), gate = p.z ? z * sg : 1.0f;
        const float dy = act_load<T>(q.dy, r * q.dy_ld + c, p.rows * q.dy_ld), w = p.w[c];
        const float v = p.before ? x : x * gate, dn = dy * w * (p.before ? gate : 1.0f);
        const float dv = rs * (dn - v * k);
        act_store<T>(q.dx, r * q.dx_ld + c, p.rows * q.dx_ld, p.before ? dv : dv * gate);
        if (p.z) {
          const float dg = p.before ? dy * v * rs * w : dv * x;
          act_store<T>(q.dz, r * q.dz_ld + c, p.rows * q.dz_ld, dg * sg * (1.0f + z * (1.0f - sg)));
        }
        part[c] += dy * v * rs * (p.before ? gate : 1.0f);
      }
    }
}

template <typename T, typename R> __global__ void add_norm_fwd_kernel(const AddNormParams p) {
  __shared__ float s[32];
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    float rx = 1.0f;
    if (p.post) {
      float ss = 0.0f;
      for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld);
        ss = fmaf(x, x, ss);
      }
      rx = rsqrtf(cta_sum(ss, s) / (float)p.d + p.eps);
    }
    float ss = 0.0f;
    for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
      float v = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld);
      if (p.post) v *= rx * p.post[c];
      if (p.scale) v *= p.scale[c];
      if (p.res) v += act_load<R>(p.res, r * p.res_ld + c, p.rows * p.res_ld);
      act_store<R>(p.res_out, r * p.ro_ld + c, p.rows * p.ro_ld, v);
      if constexpr (sizeof(R) == 2) v = __bfloat162float(__float2bfloat16_rn(v));
      ss = fmaf(v, v, ss);
    }
    const float rs = rsqrtf(cta_sum(ss, s) / (float)p.d + p.eps);
    for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads)
      act_store<T>(p.y, r * p.y_ld + c, p.rows * p.y_ld,
                   act_load<R>(p.res_out, r * p.ro_ld + c, p.rows * p.ro_ld) * rs * p.w[c]);
  }
}

template <typename T, typename R> __global__ void add_norm_bwd_kernel(const AddNormBwdParams q) {
  __shared__ float s[32];
  const AddNormParams &p = q.f;
  float *part = q.part + blockIdx.x * 3 * p.d;
  for (int64_t c = threadIdx.x; c < 3 * p.d; c += kNormThreads) part[c] = 0.0f;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    __syncthreads();
    float ss = 0.0f, sd = 0.0f, sx = 0.0f;
    for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
      const float v = act_load<R>(p.res_out, r * p.ro_ld + c, p.rows * p.ro_ld);
      ss = fmaf(v, v, ss);
      sd = fmaf(act_load<T>(q.dy, r * q.dy_ld + c, p.rows * q.dy_ld) * p.w[c], v, sd);
      if (p.post) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld);
        sx = fmaf(x, x, sx);
      }
    }
    const float rs = rsqrtf(cta_sum(ss, s) / (float)p.d + p.eps);
    const float k = cta_sum(sd, s) * rs * rs / (float)p.d;
    const float rx = p.post ? rsqrtf(cta_sum(sx, s) / (float)p.d + p.eps) : 1.0f;
    float sp = 0.0f;
    for (int pass = p.post ? 0 : 1; pass < 2; ++pass) {
      const float kx = pass && p.post ? cta_sum(sp, s) * rx * rx / (float)p.d : 0.0f;
      for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
        const float v = act_load<R>(p.res_out, r * p.ro_ld + c, p.rows * p.ro_ld);
        const float dy = act_load<T>(q.dy, r * q.dy_ld + c, p.rows * q.dy_ld);
        float dr = rs * (dy * p.w[c] - v * k);
        if (q.dro) dr += act_load<R>(q.dro, r * q.dro_ld + c, p.rows * q.dro_ld);
        const float x = (p.post || p.scale) ? act_load<T>(p.x, r * p.x_ld + c, p.rows * p.x_ld) : 0.0f;
        const float dv = p.scale ? dr * p.scale[c] : dr;
        const float dn = p.post ? dv * p.post[c] : dv;
        if (!pass) {
          sp = fmaf(dn, x, sp);
          continue;
        }
        if (q.dres) act_store<R>(q.dres, r * q.dres_ld + c, p.rows * q.dres_ld, dr);
        act_store<T>(q.dx, r * q.dx_ld + c, p.rows * q.dx_ld, p.post ? rx * (dn - x * kx) : dn);
        part[c] += dy * v * rs;
        if (p.post) part[p.d + c] += dv * x * rx;
        if (p.scale) part[2 * p.d + c] += dr * (p.post ? x * rx * p.post[c] : x);
      }
    }
  }
}

}  // namespace ssm
