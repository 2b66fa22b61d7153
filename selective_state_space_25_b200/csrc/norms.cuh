// norms.cuh -- the gated RMS norm and the residual-add norm, forward and
// backward.
//
// Bound by memory (bf16 gated norm 16384 x 1536: forward 33 us, backward 60, floors 23
// and 38; add norm 32768 x 2048: 85 and 120, floors 82 and 102).  A row (of a group, for the grouped norm) is held in registers
// by TPR threads of a CTA, VPT vectors of E elements each (16 bytes of the
// activations), so every input is read once and every output written once; the
// sums go over shuffles and, above a warp, one shared-memory exchange.  TPR is a
// power of two from 8 to 512, chosen with VPT to leave the fewest idle threads
// (norm_plan).  Backward, a CTA walks rows and its threads keep their columns'
// sums of the parameters' gradients in registers; each CTA writes one partial row.
// Rows longer than that (512 threads of 4 vectors; of 3 in the add norm's backward
// with scale or post norm, so 6144 columns) are re-read by a CTA of 256 threads (that
// backward at 8192 x 8192: 1485 us, 12 % of the copy bandwidth).
#pragma once

#include "block_common.cuh"

namespace ssm {

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
  int tpr;     // threads of a row
};
struct GatedNormBwdParams {
  GatedNormParams f;
  const void *dy;
  int64_t dy_ld;
  void *dx, *dz;
  int64_t dx_ld, dz_ld;
  int parts;
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
  int tpr;
};
struct AddNormBwdParams {
  AddNormParams f;  // res_out is read
  const void *dy, *dro;
  int64_t dy_ld, dro_ld;
  void *dx, *dres;
  int64_t dx_ld, dres_ld;
  int parts;
  float *part;  // (parts, 3, d): dweight, dpost_weight, dscale
};

// Elements of a vector backward, where the rows in flight, the next ones and the
// parameters' sums share the registers (forward: 16 bytes of the activations).
constexpr int kNormBwdElems = 4;
constexpr int kNormThreads = 256;   // of a CTA, when a row takes no more
constexpr int kNormMaxTpr = 512;    // at most 128 registers a thread then

// E elements as loaded: registers for what is in flight, unpacked to fp32 where
// they are used.
template <typename T, int E> struct RawElems {
  static constexpr int kWords = E * sizeof(T) == 32 ? 2 : 1, kPer = E / kWords;
  typename VecWord<T, kPer>::type w[kWords];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = {};
  }
  // E elements at q, inside the buffer of n elements from lo on
  __device__ __forceinline__ void load(const T *q, const void *lo, int64_t n) {
    using W = typename VecWord<T, kPer>::type;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      if (in_bounds(q + k * kPer - static_cast<const T *>(lo), n - (kPer - 1), kBndAct))
        w[k] = *reinterpret_cast<const W *>(q + k * kPer);
  }
  __device__ __forceinline__ void get(float *v) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) unpack(w[k], v + k * kPer);
  }
  __device__ __forceinline__ void get(float2 *v) const {
    float f[E];
    get(f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
  }
};
template <typename T, int E>
__device__ __forceinline__ void st_elems(T *q, void *lo, int64_t n, const float *v) {
  using Raw = RawElems<T, E>;
  const int64_t i = q - static_cast<T *>(lo);
#pragma unroll
  for (int k = 0; k < Raw::kWords; ++k)
    if (in_bounds(i + k * Raw::kPer, n - (Raw::kPer - 1), kBndAct))
      st_vec<T, Raw::kPer>(q, k * Raw::kPer, E, v + k * Raw::kPer);
}
template <typename T, int E>
__device__ __forceinline__ void st_elems(T *q, void *lo, int64_t n, const float2 *v) {
  float f[E];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) f[2 * e] = v[e].x, f[2 * e + 1] = v[e].y;
  st_elems<T, E>(q, lo, n, f);
}
// A thread's place in a row: its pointer there; one past nothing where lo is NULL.
template <typename T>
__device__ __forceinline__ T *row_at(const void *lo, int64_t r, int64_t ld, int64_t c) {
  return const_cast<T *>(static_cast<const T *>(lo)) + (r * ld + c);
}
// E parameters of columns c .. c + E - 1.
template <int E>
__device__ __forceinline__ void ld_params(const float *p, int c, int64_t d, float *v) {
  if (!in_bounds(c, d - (E - 1), kBndParam)) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 1.0f;
  } else if constexpr (E % 4 == 0) {
#pragma unroll
    for (int e = 0; e < E; e += 4) unpack(__ldg(reinterpret_cast<const float4 *>(p + c + e)), v + e);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __ldg(p + c + e);
  }
}

template <int E>
__device__ __forceinline__ void ld_params(const float *p, int c, int64_t d, float2 *v) {
  float f[E];
  ld_params<E>(p, c, d, f);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
}

// Sums of N values over the tpr threads of a row, the same in each of them.
// buf: one of two buffers taken in turn, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float (*buf)[N]) {
  // o = 4, 2, 1 always (tpr >= 8); 8 and 16 within wider rows
  if (tpr > 16)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], 16);
  if (tpr > 8)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], 8);
#pragma unroll
  for (int o = 4; o > 0; o /= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  if (tpr <= 32) return;
  const int warp = threadIdx.x / 32, warps = tpr / 32;
  if (threadIdx.x % 32 == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) buf[warp][k] = v[k];
  __syncthreads();
  const int first = warp / warps * warps;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.0f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += buf[first + w][k];
}

// Element e of values kept as pairs.
__device__ __forceinline__ float at(const float *v, int e) { return v[e]; }
__device__ __forceinline__ float at(const float2 *v, int e) { return e % 2 ? v[e / 2].y : v[e / 2].x; }

// How the gate meets the norm.
enum GateForm { kNoGate, kGateFirst, kNormFirst };

// ------------------------------------------------------- gated norm forward
template <typename T, int E, int VPT, int FORM>
__global__ void __launch_bounds__(kNormMaxTpr) gated_norm_fwd_kernel(const GatedNormParams p) {
  __shared__ float buf[32][1];
  const int64_t n = p.d / p.groups;
  const int nv = (int)(n / E);
  const float inv = 1.0f / (float)n;
  const int slot = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
  const int64_t k = blockIdx.x * (int64_t)(blockDim.x / p.tpr) + slot;
  const bool on = k < p.rows * p.groups;
  const int64_t r = p.groups == 1 ? k : k / p.groups, c0 = (k - r * p.groups) * n;
  const int64_t xn = extent(p.rows, p.d, p.x_ld), zn = extent(p.rows, p.d, p.z_ld);
  RawElems<T, E> x[VPT], z[FORM != kNoGate ? VPT : 1];
  const int hop = p.tpr * E;  // elements between a thread's vectors
  const T *px = row_at<T>(p.x, r, p.x_ld, c0 + lane * E), *pz = row_at<T>(p.z, r, p.z_ld, c0 + lane * E);
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    x[q].clear();
    if constexpr (FORM != kNoGate) z[q].clear();
    if (on && lane + q * p.tpr < nv) {
      x[q].load(px + q * hop, p.x, xn);
      if constexpr (FORM != kNoGate) z[q].load(pz + q * hop, p.z, zn);
    }
  }
  using F = typename Lanes<E>::F;
  constexpr int N = Lanes<E>::N;
  F g[FORM != kNoGate ? VPT : 1][N];  // x silu(z), or silu(z) with the norm first
  F ss = bc<F>(0.0f);
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    F v[N];
    x[q].get(v);
    if constexpr (FORM != kNoGate) {
      z[q].get(g[q]);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        g[q][e] = mulv(g[q][e], sigmoidv(g[q][e]));
        if (FORM == kGateFirst) v[e] = g[q][e] = mulv(g[q][e], v[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) ss = fmav(v[e], v[e], ss);
  }
  float s[1] = {hsum(ss)};
  row_sum<1>(s, p.tpr, buf);
  const float rs = rsqrtf(fmaf(s[0], inv, p.eps));
  T *py = row_at<T>(p.y, r, p.y_ld, c0 + lane * E);
  const int64_t yn = extent(p.rows, p.d, p.y_ld);
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    if (!on || lane + q * p.tpr >= nv) continue;
    F w[N], v[N];
    ld_params<E>(p.w + c0, lane * E + q * hop, n, w);
    if constexpr (FORM != kGateFirst) x[q].get(v);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if constexpr (FORM == kGateFirst)
        v[e] = mulv(g[q][e], mulv(w[e], rs));
      else
        v[e] = mulv(v[e], mulv(w[e], rs));
      if constexpr (FORM == kNormFirst) v[e] = mulv(v[e], g[q][e]);
    }
    st_elems<T, E>(py + q * hop, p.y, yn, v);
  }
}

// ------------------------------------------------------ gated norm backward
// With n = v rs the normed value (v = x or x silu(z)) and dn its gradient:
//   dv = rs (dn - n mean(dn n)).
// CTA b works on group b % groups; the next row's loads are issued before a row's
// sums are waited for.
template <typename T, int E, int VPT, int FORM>
__global__ void __launch_bounds__(kNormMaxTpr) gated_norm_bwd_kernel(const GatedNormBwdParams q_) {
  const GatedNormParams &p = q_.f;
  constexpr bool GATE = FORM != kNoGate;
  __shared__ float buf[2][32][2];
  extern __shared__ float red[];  // (slots, n)
  const int64_t n = p.d / p.groups;
  const int nv = (int)(n / E);
  const float inv = 1.0f / (float)n;
  const int slots = blockDim.x / p.tpr, slot = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
  const int64_t grp = blockIdx.x % (unsigned)p.groups, blk = blockIdx.x / (unsigned)p.groups;
  const int64_t c0 = grp * n;
  const int64_t xn = extent(p.rows, p.d, p.x_ld), zn = extent(p.rows, p.d, p.z_ld),
                gn = extent(p.rows, p.d, q_.dy_ld), dxn = extent(p.rows, p.d, q_.dx_ld),
                dzn = extent(p.rows, p.d, q_.dz_ld);
  using F = typename Lanes<E>::F;
  constexpr int N = Lanes<E>::N;
  F dw[VPT][N];
#pragma unroll
  for (int q = 0; q < VPT; ++q)
#pragma unroll
    for (int e = 0; e < N; ++e) dw[q][e] = bc<F>(0.0f);
  RawElems<T, E> nx[VPT], ng[VPT], nz[GATE ? VPT : 1];
  const int hop = p.tpr * E;                     // elements between a thread's vectors
  const int64_t step = q_.parts * (int64_t)slots;  // rows between a slot's
  const int64_t r0 = blk * slots + slot, cl = c0 + lane * E;
  const T *px = row_at<T>(p.x, r0, p.x_ld, cl), *pz = row_at<T>(p.z, r0, p.z_ld, cl),
          *pg = row_at<T>(q_.dy, r0, q_.dy_ld, cl);
  T *pdx = row_at<T>(q_.dx, r0, q_.dx_ld, cl), *pdz = row_at<T>(q_.dz, r0, q_.dz_ld, cl);
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      nx[q].clear();
      ng[q].clear();
      if constexpr (GATE) nz[q].clear();
      if (r < p.rows && lane + q * p.tpr < nv) {
        nx[q].load(px + q * hop, p.x, xn);
        ng[q].load(pg + q * hop, q_.dy, gn);
        if constexpr (GATE) nz[q].load(pz + q * hop, p.z, zn);
      }
    }
    px += step * p.x_ld;
    pg += step * q_.dy_ld;
    if constexpr (GATE) pz += step * p.z_ld;
  };
  int turn = 0;
  load(r0);
  for (int64_t base = blk * slots; base < p.rows; base += step) {
    const int64_t r = base + slot;
    const bool on = r < p.rows;
    RawElems<T, E> rx[VPT], rg[VPT], rz[GATE ? VPT : 1];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      rx[q] = nx[q];
      rg[q] = ng[q];
      if constexpr (GATE) rz[q] = nz[q];
    }
    load(r + step);
    F s0 = bc<F>(0.0f), s1 = s0;
    F sg[GATE ? VPT : 1][N];  // sigmoid(z)
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      F v[N], dn[N], w[N], z[N];
      ld_params<E>(p.w + c0, j < nv ? lane * E + q * hop : 0, n, w);
      rx[q].get(v);
      rg[q].get(dn);
      if constexpr (GATE) rz[q].get(z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        dn[e] = mulv(dn[e], w[e]);
        if constexpr (GATE) {
          sg[q][e] = sigmoidv(z[e]);
          const F gate = mulv(z[e], sg[q][e]);
          if (FORM == kNormFirst)
            dn[e] = mulv(dn[e], gate);
          else
            v[e] = mulv(v[e], gate);
        }
        s0 = fmav(v[e], v[e], s0);
        s1 = fmav(dn[e], v[e], s1);
      }
    }
    float s[2] = {hsum(s0), hsum(s1)};
    row_sum<2>(s, p.tpr, buf[turn]);
    turn ^= 1;
    const float rs = rsqrtf(fmaf(s[0], inv, p.eps));
    const float k = s[1] * rs * rs * inv;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      if (!on || j >= nv) continue;
      F x[N], dy[N], z[N], w[N], dx[N], dz[N];
      ld_params<E>(p.w + c0, lane * E + q * hop, n, w);
      rx[q].get(x);
      rg[q].get(dy);
      if constexpr (GATE) rz[q].get(z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        F v = x[e], dn = mulv(dy[e], w[e]), gate, ds;
        if constexpr (GATE) {
          gate = mulv(z[e], sg[q][e]);
          // silu'(z) = s + z s (1 - s)
          ds = fmav(gate, fmav(sg[q][e], bc<F>(-1.0f), bc<F>(1.0f)), sg[q][e]);
          if (FORM == kNormFirst)
            dn = mulv(dn, gate);
          else
            v = mulv(v, gate);
        }
        const F dv = mulv(fmav(v, bc<F>(-k), dn), bc<F>(rs)), nr = mulv(v, bc<F>(rs));
        if constexpr (FORM == kNormFirst) {
          const F gy = mulv(dy[e], nr);
          dx[e] = dv;
          dz[e] = mulv(mulv(gy, w[e]), ds);
          dw[q][e] = fmav(gy, gate, dw[q][e]);
        } else {
          dx[e] = dv;
          if constexpr (GATE) {
            dx[e] = mulv(dv, gate);
            dz[e] = mulv(mulv(dv, x[e]), ds);
          }
          dw[q][e] = fmav(dy[e], nr, dw[q][e]);
        }
      }
      st_elems<T, E>(pdx + q * hop, q_.dx, dxn, dx);
      if constexpr (GATE) st_elems<T, E>(pdz + q * hop, q_.dz, dzn, dz);
    }
    pdx += step * q_.dx_ld;
    if constexpr (GATE) pdz += step * q_.dz_ld;
  }
  // the columns' sums over the CTA's slots, in order
  float *part = q_.part + blk * p.d;
  if (slots > 1) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      if (j < nv)
#pragma unroll
        for (int e = 0; e < E; ++e) red[slot * n + j * E + e] = at(dw[q], e);
    }
    __syncthreads();
    for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
      float t = red[c];
      for (int k = 1; k < slots; ++k) t += red[k * n + c];
      if (in_bounds(c0 + c, p.d, kBndWork)) part[c0 + c] = t;
    }
  } else {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      if (j < nv)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (in_bounds(c0 + j * E + e, p.d, kBndWork)) part[c0 + j * E + e] = at(dw[q], e);
    }
  }
}

// --------------------------------------------------------- add norm forward
template <typename R> __device__ __forceinline__ float round_to(float v) {
  if constexpr (sizeof(R) == 2) return __bfloat162float(__float2bfloat16_rn(v));
  return v;
}

template <typename T, typename R, int E, int VPT>
__global__ void __launch_bounds__(kNormMaxTpr) add_norm_fwd_kernel(const AddNormParams p) {
  __shared__ float buf[2][32][1];
  const int nv = (int)(p.d / E);
  const float inv = 1.0f / (float)p.d;
  const int slot = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
  const int64_t r = blockIdx.x * (int64_t)(blockDim.x / p.tpr) + slot;
  const bool on = r < p.rows;
  const int64_t xn = extent(p.rows, p.d, p.x_ld), rn = extent(p.rows, p.d, p.res_ld);
  RawElems<T, E> rx[VPT];
  RawElems<R, E> ro[VPT];
  const int hop = p.tpr * E;  // elements between a thread's vectors
  const T *px = row_at<T>(p.x, r, p.x_ld, lane * E);
  const R *pr = row_at<R>(p.res, r, p.res_ld, lane * E);
  R *po = row_at<R>(p.res_out, r, p.ro_ld, lane * E);
  T *py = row_at<T>(p.y, r, p.y_ld, lane * E);
  const int64_t on_ = extent(p.rows, p.d, p.ro_ld), yn = extent(p.rows, p.d, p.y_ld);
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    rx[q].clear();
    ro[q].clear();
    if (on && lane + q * p.tpr < nv) {
      rx[q].load(px + q * hop, p.x, xn);
      if (p.res) ro[q].load(pr + q * hop, p.res, rn);
    }
  }
  float rxs = 1.0f, s[1] = {0.0f};
  if (p.post) {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      float v[E];
      rx[q].get(v);
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] = fmaf(v[e], v[e], s[0]);
    }
    row_sum<1>(s, p.tpr, buf[1]);
    rxs = rsqrtf(fmaf(s[0], inv, p.eps));
    s[0] = 0.0f;
  }
  float v[VPT][E];
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int j = lane + q * p.tpr;
    float o[E], w[E];
    rx[q].get(v[q]);
    ro[q].get(o);
    if (p.post) {
      ld_params<E>(p.post, j < nv ? lane * E + q * hop : 0, p.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) v[q][e] *= rxs * w[e];
    }
    if (p.scale) {
      ld_params<E>(p.scale, j < nv ? lane * E + q * hop : 0, p.d, w);
#pragma unroll
      for (int e = 0; e < E; ++e) v[q][e] *= w[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[q][e] = round_to<R>(p.res ? v[q][e] + o[e] : v[q][e]);
      s[0] = fmaf(v[q][e], v[q][e], s[0]);
    }
    if (on && j < nv)
      st_elems<R, E>(po + q * hop, p.res_out, on_, v[q]);
  }
  row_sum<1>(s, p.tpr, buf[0]);
  const float rs = rsqrtf(fmaf(s[0], inv, p.eps));
#pragma unroll
  for (int q = 0; q < VPT; ++q) {
    const int j = lane + q * p.tpr;
    if (!on || j >= nv) continue;
    float w[E];
    ld_params<E>(p.w, lane * E + q * hop, p.d, w);
#pragma unroll
    for (int e = 0; e < E; ++e) v[q][e] *= rs * w[e];
    st_elems<T, E>(py + q * hop, p.y, yn, v[q]);
  }
}

// -------------------------------------------------------- add norm backward
// dr = rs (dy w - n mean(dy w n)) + dresidual_out, n = r rs;  dscale += dr v;
// dv = dr scale;  with the post norm (xn = x rx, v = xn post): dpost += dv xn,
// dx = rx (dv post - xn mean(dv post xn)), else dx = dv.
template <typename T, typename R, int E, int VPT, bool POST, bool SCALE>
__global__ void __launch_bounds__(kNormMaxTpr) add_norm_bwd_kernel(const AddNormBwdParams q_) {
  const AddNormParams &p = q_.f;
  constexpr bool X = POST || SCALE;
  __shared__ float buf[2][32][3];
  __shared__ float buf2[2][32][1];
  extern __shared__ float red[];  // (slots, d)
  const int nv = (int)(p.d / E);
  const float inv = 1.0f / (float)p.d;
  const int slots = blockDim.x / p.tpr, slot = threadIdx.x / p.tpr, lane = threadIdx.x % p.tpr;
  const int64_t ron = extent(p.rows, p.d, p.ro_ld), gn = extent(p.rows, p.d, q_.dy_ld),
                xn = extent(p.rows, p.d, p.x_ld), drn = extent(p.rows, p.d, q_.dro_ld),
                dxn = extent(p.rows, p.d, q_.dx_ld), don = extent(p.rows, p.d, q_.dres_ld);
  using F = typename Lanes<E>::F;
  constexpr int N = Lanes<E>::N;
  F dw[VPT][N], dp[POST ? VPT : 1][N], dsc[SCALE ? VPT : 1][N];
#pragma unroll
  for (int q = 0; q < VPT; ++q)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      dw[q][e] = bc<F>(0.0f);
      if constexpr (POST) dp[q][e] = bc<F>(0.0f);
      if constexpr (SCALE) dsc[q][e] = bc<F>(0.0f);
    }
  RawElems<R, E> nv_[VPT], nd[VPT];
  RawElems<T, E> ng[VPT], nx[X ? VPT : 1];
  const int hop = p.tpr * E;                       // elements between a thread's vectors
  const int64_t step = q_.parts * (int64_t)slots;  // rows between a slot's
  const int64_t r0 = blockIdx.x * (int64_t)slots + slot;
  const R *pv = row_at<R>(p.res_out, r0, p.ro_ld, lane * E), *pd = row_at<R>(q_.dro, r0, q_.dro_ld, lane * E);
  const T *pg = row_at<T>(q_.dy, r0, q_.dy_ld, lane * E), *px = row_at<T>(p.x, r0, p.x_ld, lane * E);
  T *pdx = row_at<T>(q_.dx, r0, q_.dx_ld, lane * E);
  R *pdr = row_at<R>(q_.dres, r0, q_.dres_ld, lane * E);
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      nv_[q].clear();
      nd[q].clear();
      ng[q].clear();
      if constexpr (X) nx[q].clear();
      if (r < p.rows && lane + q * p.tpr < nv) {
        nv_[q].load(pv + q * hop, p.res_out, ron);
        ng[q].load(pg + q * hop, q_.dy, gn);
        if (q_.dro) nd[q].load(pd + q * hop, q_.dro, drn);
        if constexpr (X) nx[q].load(px + q * hop, p.x, xn);
      }
    }
    pv += step * p.ro_ld;
    pg += step * q_.dy_ld;
    pd += step * q_.dro_ld;
    if constexpr (X) px += step * p.x_ld;
  };
  int turn = 0;
  load(r0);
  for (int64_t base = blockIdx.x * (int64_t)slots; base < p.rows; base += step) {
    const int64_t r = base + slot;
    const bool on = r < p.rows;
    RawElems<R, E> rv[VPT], rd[VPT];
    RawElems<T, E> rg[VPT], rx_[X ? VPT : 1];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      rv[q] = nv_[q];
      rd[q] = nd[q];
      rg[q] = ng[q];
      if constexpr (X) rx_[q] = nx[q];
    }
    load(r + step);
    F s0 = bc<F>(0.0f), s1 = s0, s2 = s0;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      F w[N], v[N], g[N];
      ld_params<E>(p.w, j < nv ? lane * E + q * hop : 0, p.d, w);
      rv[q].get(v);
      rg[q].get(g);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s0 = fmav(v[e], v[e], s0);
        s1 = fmav(mulv(g[e], w[e]), v[e], s1);
      }
      if constexpr (POST) {
        rx_[q].get(v);
#pragma unroll
        for (int e = 0; e < N; ++e) s2 = fmav(v[e], v[e], s2);
      }
    }
    float s[3] = {hsum(s0), hsum(s1), hsum(s2)};
    row_sum<3>(s, p.tpr, buf[turn]);
    // Without x the two divisions are left to be made here: the compiler then keeps
    // the next row's loads in front of the sums (bf16, 32768 x 2048: 120 us, 163 with
    // products by the inverse, whose loads sink to their use); with x the products
    // are faster (16384 x 768, scale and post norm: 61 us, 66).
    // A place without a row holds zeros, which add nothing to the columns' sums while
    // its inverse roots are finite: not those of eps = 0.
    const float eps = on ? p.eps : 1.0f;
    const float rs = rsqrtf(X ? fmaf(s[0], inv, eps) : s[0] / (float)p.d + eps);
    const float mean = X ? s[1] * inv : s[1] / (float)p.d;
    const F k = bc<F>(-mean * rs * rs * rs), rsv = bc<F>(rs);
    const float rx = POST ? rsqrtf(fmaf(s[2], inv, eps)) : 1.0f;
    F sp = bc<F>(0.0f), dv[VPT][N];
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      const int cj = j < nv ? lane * E + q * hop : 0;
      F w[N], v[N], g[N], x[N];
      ld_params<E>(p.w, cj, p.d, w);
      rv[q].get(v);
      rg[q].get(g);
      rd[q].get(dv[q]);
      if constexpr (X) rx_[q].get(x);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const F gr = mulv(g[e], rsv);
        dv[q][e] = fmav(gr, w[e], fmav(v[e], k, dv[q][e]));
        dw[q][e] = fmav(gr, v[e], dw[q][e]);
      }
      if (q_.dres && on && j < nv) st_elems<R, E>(pdr + q * hop, q_.dres, don, dv[q]);
      if constexpr (POST) {
        ld_params<E>(p.post, cj, p.d, w);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = mulv(x[e], bc<F>(rx));  // xn
      }
      if constexpr (SCALE) {
        F sc[N];
        ld_params<E>(p.scale, cj, p.d, sc);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          dsc[q][e] = fmav(dv[q][e], POST ? mulv(x[e], w[e]) : x[e], dsc[q][e]);
          dv[q][e] = mulv(dv[q][e], sc[e]);
        }
      }
      if constexpr (POST) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          dp[q][e] = fmav(dv[q][e], x[e], dp[q][e]);
          dv[q][e] = mulv(dv[q][e], w[e]);
          sp = fmav(dv[q][e], x[e], sp);
        }
      }
    }
    F kx = bc<F>(0.0f);
    if constexpr (POST) {
      float t[1] = {hsum(sp)};
      row_sum<1>(t, p.tpr, buf2[turn]);
      kx = bc<F>(-t[0] * inv);
    }
    turn ^= 1;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
      const int j = lane + q * p.tpr;
      if (!on || j >= nv) continue;
      if constexpr (POST) {
        F x[N];
        rx_[q].get(x);
#pragma unroll
        for (int e = 0; e < N; ++e) dv[q][e] = mulv(fmav(mulv(x[e], bc<F>(rx)), kx, dv[q][e]), bc<F>(rx));
      }
      st_elems<T, E>(pdx + q * hop, q_.dx, dxn, dv[q]);
    }
    pdx += step * q_.dx_ld;
    pdr += step * q_.dres_ld;
  }
  float *part = q_.part + blockIdx.x * 3 * p.d;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if ((k == 1 && !POST) || (k == 2 && !SCALE)) continue;
    const auto sum = [&](int q, int e) {
      if constexpr (POST)
        if (k == 1) return at(dp[q], e);
      if constexpr (SCALE)
        if (k == 2) return at(dsc[q], e);
      return at(dw[q], e);
    };
    if (slots > 1) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int j = lane + q * p.tpr;
        if (j < nv)
#pragma unroll
          for (int e = 0; e < E; ++e) red[slot * p.d + j * E + e] = sum(q, e);
      }
      __syncthreads();
      for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
        float t = red[c];
        for (int z = 1; z < slots; ++z) t += red[z * p.d + c];
        if (in_bounds(c, p.d, kBndWork)) part[k * p.d + c] = t;
      }
    } else {
#pragma unroll
      for (int q = 0; q < VPT; ++q) {
        const int j = lane + q * p.tpr;
        if (j < nv)
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (in_bounds(j * E + e, p.d, kBndWork)) part[k * p.d + j * E + e] = sum(q, e);
      }
    }
  }
}

// ------------------------------------------------------------- longer rows
// A CTA of 256 threads a row (of a group), which is read again for the second
// pass; the parameters' sums are kept in the CTA's partial row.
template <typename T>
__device__ __forceinline__ float act_load(const void *p, int64_t i, int64_t n) {
  return in_bounds(i, n, kBndAct) ? Elem<T>::load(static_cast<const T *>(p), i) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void act_store(void *p, int64_t i, int64_t n, float v) {
  if (in_bounds(i, n, kBndAct)) Elem<T>::store(static_cast<T *>(p), i, v);
}

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

template <typename T> __global__ void gated_norm_fwd_long_kernel(const GatedNormParams p) {
  __shared__ float s[32];
  const int64_t n = p.d / p.groups, xn = extent(p.rows, p.d, p.x_ld),
                zn = extent(p.rows, p.d, p.z_ld), yn = extent(p.rows, p.d, p.y_ld);
  for (int64_t k = blockIdx.x; k < p.rows * p.groups; k += gridDim.x) {
    const int64_t r = k / p.groups, c0 = k % p.groups * n;
    float ss = 0.0f;
    for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
      float v = act_load<T>(p.x, r * p.x_ld + c, xn);
      if (p.z && !p.before) v *= silu_f32(act_load<T>(p.z, r * p.z_ld + c, zn));
      ss = fmaf(v, v, ss);
    }
    const float rs = rsqrtf(cta_sum(ss, s) / (float)n + p.eps);
    for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
      float v = act_load<T>(p.x, r * p.x_ld + c, xn) * rs * p.w[c];
      if (p.z) v *= silu_f32(act_load<T>(p.z, r * p.z_ld + c, zn));
      act_store<T>(p.y, r * p.y_ld + c, yn, v);
    }
  }
}

template <typename T> __global__ void gated_norm_bwd_long_kernel(const GatedNormBwdParams q) {
  __shared__ float s[32];
  const GatedNormParams &p = q.f;
  const int64_t n = p.d / p.groups, xn = extent(p.rows, p.d, p.x_ld),
                zn = extent(p.rows, p.d, p.z_ld), gn = extent(p.rows, p.d, q.dy_ld),
                dxn = extent(p.rows, p.d, q.dx_ld), dzn = extent(p.rows, p.d, q.dz_ld);
  float *part = q.part + blockIdx.x * p.d;
  for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) part[c] = 0.0f;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x)
    for (int64_t c0 = 0; c0 < p.d; c0 += n) {
      __syncthreads();
      float ss = 0.0f, sd = 0.0f;
      for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, xn);
        const float gate = p.z ? silu_f32(act_load<T>(p.z, r * p.z_ld + c, zn)) : 1.0f;
        const float dy = act_load<T>(q.dy, r * q.dy_ld + c, gn);
        const float v = p.before ? x : x * gate, dn = dy * p.w[c] * (p.before ? gate : 1.0f);
        ss = fmaf(v, v, ss);
        sd = fmaf(dn, v, sd);
      }
      const float rs = rsqrtf(cta_sum(ss, s) / (float)n + p.eps);
      const float k = cta_sum(sd, s) * rs * rs / (float)n;
      for (int64_t c = c0 + threadIdx.x; c < c0 + n; c += kNormThreads) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, xn);
        const float z = p.z ? act_load<T>(p.z, r * p.z_ld + c, zn) : 0.0f;
        const float sg = sigmoid_f32(z), gate = p.z ? z * sg : 1.0f;
        const float dy = act_load<T>(q.dy, r * q.dy_ld + c, gn), w = p.w[c];
        const float v = p.before ? x : x * gate, dn = dy * w * (p.before ? gate : 1.0f);
        const float dv = rs * (dn - v * k);
        act_store<T>(q.dx, r * q.dx_ld + c, dxn, p.before ? dv : dv * gate);
        if (p.z) {
          const float dg = p.before ? dy * v * rs * w : dv * x;
          act_store<T>(q.dz, r * q.dz_ld + c, dzn, dg * sg * (1.0f + z * (1.0f - sg)));
        }
        part[c] += dy * v * rs * (p.before ? gate : 1.0f);
      }
    }
}

template <typename T, typename R> __global__ void add_norm_fwd_long_kernel(const AddNormParams p) {
  __shared__ float s[32];
  const int64_t xn = extent(p.rows, p.d, p.x_ld), rn = extent(p.rows, p.d, p.res_ld),
                on = extent(p.rows, p.d, p.ro_ld), yn = extent(p.rows, p.d, p.y_ld);
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    float rx = 1.0f;
    if (p.post) {
      float ss = 0.0f;
      for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, xn);
        ss = fmaf(x, x, ss);
      }
      rx = rsqrtf(cta_sum(ss, s) / (float)p.d + p.eps);
    }
    float ss = 0.0f;
    for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
      float v = act_load<T>(p.x, r * p.x_ld + c, xn);
      if (p.post) v *= rx * p.post[c];
      if (p.scale) v *= p.scale[c];
      if (p.res) v += act_load<R>(p.res, r * p.res_ld + c, rn);
      v = round_to<R>(v);
      act_store<R>(p.res_out, r * p.ro_ld + c, on, v);
      ss = fmaf(v, v, ss);
    }
    const float rs = rsqrtf(cta_sum(ss, s) / (float)p.d + p.eps);
    for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads)
      act_store<T>(p.y, r * p.y_ld + c, yn, act_load<R>(p.res_out, r * p.ro_ld + c, on) * rs * p.w[c]);
  }
}

template <typename T, typename R> __global__ void add_norm_bwd_long_kernel(const AddNormBwdParams q) {
  __shared__ float s[32];
  const AddNormParams &p = q.f;
  const int64_t xn = extent(p.rows, p.d, p.x_ld), on = extent(p.rows, p.d, p.ro_ld),
                gn = extent(p.rows, p.d, q.dy_ld), drn = extent(p.rows, p.d, q.dro_ld),
                dxn = extent(p.rows, p.d, q.dx_ld), dsn = extent(p.rows, p.d, q.dres_ld);
  float *part = q.part + blockIdx.x * 3 * p.d;
  for (int64_t c = threadIdx.x; c < 3 * p.d; c += kNormThreads) part[c] = 0.0f;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    __syncthreads();
    float ss = 0.0f, sd = 0.0f, sx = 0.0f;
    for (int64_t c = threadIdx.x; c < p.d; c += kNormThreads) {
      const float v = act_load<R>(p.res_out, r * p.ro_ld + c, on);
      ss = fmaf(v, v, ss);
      sd = fmaf(act_load<T>(q.dy, r * q.dy_ld + c, gn) * p.w[c], v, sd);
      if (p.post) {
        const float x = act_load<T>(p.x, r * p.x_ld + c, xn);
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
        const float v = act_load<R>(p.res_out, r * p.ro_ld + c, on);
        const float dy = act_load<T>(q.dy, r * q.dy_ld + c, gn);
        float dr = rs * (dy * p.w[c] - v * k);
        if (q.dro) dr += act_load<R>(q.dro, r * q.dro_ld + c, drn);
        const float x = (p.post || p.scale) ? act_load<T>(p.x, r * p.x_ld + c, xn) : 0.0f;
        const float dv = p.scale ? dr * p.scale[c] : dr;
        const float dn = p.post ? dv * p.post[c] : dv;
        if (!pass) {
          sp = fmaf(dn, x, sp);
          continue;
        }
        if (q.dres) act_store<R>(q.dres, r * q.dres_ld + c, dsn, dr);
        act_store<T>(q.dx, r * q.dx_ld + c, dxn, p.post ? rx * (dn - x * kx) : dn);
        part[c] += dy * v * rs;
        if (p.post) part[p.d + c] += dv * x * rx;
        if (p.scale) part[2 * p.d + c] += dr * (p.post ? x * rx * p.post[c] : x);
      }
    }
  }
}

}  // namespace ssm
