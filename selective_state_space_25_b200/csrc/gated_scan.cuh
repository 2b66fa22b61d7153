// gated_scan.cuh -- the gated linear recurrence: forward, backward, one-token
// step.
//
//   r = sigmoid(ga + ba), g = sigmoid(gx + bx), a = exp(A r), f = sqrt(1 - a^2)
//   h_t = a h_{t-1} + f g u          (h_t = g u where a sequence starts)
//
// Split over time.  A step is the map h -> a h + x, and maps compose: steps
// taken together are h -> P h + Q with P the product of their decays.  A CTA
// takes 32 VEC channels (128 bytes of a row) and walks tiles of kGatedChunk = 64
// steps; in a tile each of its 8 warps takes 8 steps, a lane VEC channels of
// them, and forms its decays and drives and (P, Q) in registers.  The warps'
// (P, Q) go through shared memory; each warp composes those in front of it onto
// the tile's start state and then replays its 8 steps from registers.  So every
// input is read once and nothing waits on more than 8 sequential steps, where a
// thread per channel waits on L.  Where b * d alone gives too few CTAs, up to 8
// CTAs of a cluster take consecutive tiles at once and exchange their tiles'
// (P, Q) through each other's shared memory.
//
// The adjoint is the same recurrence backwards: mu_t = a_t (dout_t + mu_{t+1}) is
// what step t hands to step t - 1, so the backward composes (P, mu) of tiles from
// the end, and recomputes the states from the tile start states that the forward
// kept (4 bytes every 64 steps and channel).
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
  int ctiles;   // CTAs across the channels
  int csize;    // CTAs of a cluster: tiles taken at once
};

struct GatedBwdParams {
  GatedParams f;  // inputs of the forward; chunk_h is read
  const void *dout;
  int64_t dout_ld;
  const float *dh_last;
  void *du, *dga, *dgx, *dz;
  int64_t du_ld, dga_ld, dgx_ld, dz_ld;
  float *dh0;
  float *part;  // (b * csize, 3, d): sums of dA, dbias_a, dbias_x
};

constexpr int kGatedWarps = 8, kGatedSteps = 8;  // warps of a CTA, steps of a warp
constexpr int kGatedThreads = 32 * kGatedWarps;
static_assert(kGatedWarps * kGatedSteps == kGatedChunk, "a tile is a chunk");
constexpr int kGatedMaxCluster = 8;
constexpr int kGatedRowBytes = 128;
// Staged bytes of a tensor's 8 rows for one warp.
constexpr int kGatedStage = kGatedSteps * kGatedRowBytes;

// Channels a lane takes: 32 VEC channels are 128 bytes.
template <typename T> constexpr int gated_vec() { return 4 / (int)sizeof(T); }

// Shared memory of a CTA that stages NT tensors two tiles deep.
constexpr int gated_smem(int nt) { return 2 * nt * kGatedWarps * kGatedStage; }

// ------------------------------------------------------------- clusters
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores v at the same shared-memory place of the cluster's CTA `rank`.
__device__ __forceinline__ void st_peer(float4 *p, int rank, float4 v) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(r), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// ------------------------------------------------------------ elementwise
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float2 rcp_2(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
__device__ __forceinline__ float2 rsqrt_2(float2 x) {
  return make_float2(rsqrt_approx(x.x), rsqrt_approx(x.y));
}
// silu of two values
__device__ __forceinline__ float2 silu_2(float2 z) {
  const float2 s = rcp_2(__fadd2_rn(ex2_2(mul2(z, f2(-kLog2e))), f2(1.0f)));
  return mul2(z, s);
}

// Composition: state after the map (P, Q) from state h.  With START a P of 0
// says that a sequence started on the way: nothing of h remains, NaN neither.
template <bool START> __device__ __forceinline__ float through(float P, float h, float Q) {
  const float r = fmaf(P, h, Q);
  return START && P == 0.0f ? Q : r;
}
// Product of two decays; with START one of 0 stays 0 beside a NaN.
template <bool START> __device__ __forceinline__ float times(float P, float a) {
  const float r = P * a;
  return START && (P == 0.0f || a == 0.0f) ? 0.0f : r;
}

// m after `front`, both (P, P, Q, Q) of a lane's channels.
template <int VEC, bool START> __device__ __forceinline__ void gated_compose(float4 &front, float4 m) {
  front.z = through<START>(m.x, front.z, m.z);
  front.x = times<START>(front.x, m.x);
  if constexpr (VEC == 2) {
    front.w = through<START>(m.y, front.w, m.w);
    front.y = times<START>(front.y, m.y);
  }
}

// Makes the tiles' compositions, which one warp of each CTA wrote, known to all
// of the cluster.  Only that warp releases at cluster scope (a release waits for
// a warp's global stores too): its release covers what the CTA's other warps
// read of the buffer two rounds ago, which the round's __syncthreads ordered
// before it.
__device__ __forceinline__ void gated_exchange(int C, bool writer) {
  if (C == 1) {
    __syncthreads();
    return;
  }
  __syncwarp();
  if (writer)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  cluster_wait();
}

// Per-lane constants: VEC channels from c0 (the pair's two for VEC = 2, one
// twice for VEC = 1).
struct GatedLane {
  float2 A2, na, nx;  // A log2 e; -bias_a log2 e; -bias_x log2 e
};
template <int VEC>
__device__ __forceinline__ float2 lane_pair(const float *p, int64_t c, int64_t d) {
  float2 v = f2(0.0f);
  if (p && c < d) v.x = ld_param(p, c, d);
  if constexpr (VEC == 2) {
    if (p && c + 1 < d) v.y = ld_param(p, c + 1, d);
  } else {
    v.y = v.x;
  }
  return v;
}
template <int VEC>
__device__ __forceinline__ GatedLane gated_lane(const GatedParams &p, int64_t c) {
  GatedLane l;
  l.A2 = mul2(lane_pair<VEC>(p.A, c, p.d), f2(kLog2e));
  l.A2 = make_float2(min_nan(l.A2.x, 126.0f), min_nan(l.A2.y, 126.0f));
  l.na = mul2(lane_pair<VEC>(p.ba, c, p.d), f2(-kLog2e));
  l.nx = mul2(lane_pair<VEC>(p.bx, c, p.d), f2(-kLog2e));
  return l;
}

// ----------------------------------------------------------------- staging
// One tensor's rows for a warp: 8 rows of 128 bytes a tile, `step` bytes to the
// next tile's.  ASYNC: 16-byte cp.async (rows 16-byte aligned, d a multiple of 16
// bytes), lane l the piece l % 8 of rows l / 8 and l / 8 + 4; else element loads.
// Rows past the end and channels past d become zeros.
template <typename T, bool ASYNC> struct GatedSrc {
  const char *p;      // the lane's first element of the next tile
  int64_t ld, step;   // bytes
  const char *lo, *hi;  // the buffer (debug-bounds build)
  __device__ __forceinline__ void init(const void *src, int64_t ld_, int64_t row, int64_t tile_rows,
                                       int64_t c0, int lane, int64_t rows, int64_t d) {
    constexpr int E = 16 / (int)sizeof(T);
    ld = ld_ * (int64_t)sizeof(T);
    step = tile_rows * ld;
    lo = static_cast<const char *>(src);
    hi = lo + extent(rows, d, ld_) * (int64_t)sizeof(T);
    p = lo + row * ld + c0 * (int64_t)sizeof(T) +
        (ASYNC ? lane / 8 * ld + lane % 8 * 16 : lane * gated_vec<T>() * (int64_t)sizeof(T));
    (void)E;
  }
  // n rows of this tile; bytes: 16 where the lane's piece lies in front of d, else
  // 0 (elements: how many of the lane's do)
  __device__ __forceinline__ void fetch(char *s, int n, int bytes, int lane) {
    if constexpr (ASYNC) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const char *q = p + 4 * j * ld;
        int b = bytes;
        if (n < kGatedSteps && lane / 8 + 4 * j >= n) b = 0;
        if (b && !in_bounds(q - lo, hi - lo - 15, kBndAct)) b = 0;
        if (n < kGatedSteps && !b) q = lo;
        cp_async16(s + j * 512 + lane * 16, q, b);
      }
    } else {
      constexpr int VEC = gated_vec<T>();
      T v[kGatedSteps][VEC];
#pragma unroll
      for (int r = 0; r < kGatedSteps; ++r)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const char *q = p + r * ld + e * (int)sizeof(T);
          v[r][e] = r < n && e < bytes && in_bounds(q - lo, hi - lo, kBndAct)
                        ? *reinterpret_cast<const T *>(q) : T(0.0f);
        }
#pragma unroll
      for (int r = 0; r < kGatedSteps; ++r)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          reinterpret_cast<T *>(s + r * kGatedRowBytes)[lane * VEC + e] = v[r][e];
    }
    p += step;
  }
};
// The `bytes` of fetch for a lane.
template <typename T, bool ASYNC>
__device__ __forceinline__ int gated_piece(int64_t c0, int lane, int64_t d) {
  if constexpr (ASYNC) return c0 + lane % 8 * (16 / (int)sizeof(T)) < d ? 16 : 0;
  const int64_t left = d - c0 - lane * gated_vec<T>();
  return left < 0 ? 0 : left < gated_vec<T>() ? (int)left : gated_vec<T>();
}

// Flat element k of a lane: step k / VEC, channel k % VEC.  Pair k of one staged
// tensor: flat elements 2 k and 2 k + 1.
template <typename T>
__device__ __forceinline__ float2 staged_pair(const char *s, int k, int lane) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(s + k * kGatedRowBytes + lane * 4);
    return make_float2(bf16lo(w), bf16hi(w));
  } else {
    const float *f = reinterpret_cast<const float *>(s) + lane;
    return make_float2(f[2 * k * 32], f[(2 * k + 1) * 32]);
  }
}

// Stores flat elements of step s: VEC channels from c.
template <typename T, bool ASYNC>
__device__ __forceinline__ void store_step(void *p, int64_t ld, int64_t row, int64_t c, int64_t d,
                                           int64_t ext, const float *v) {
  constexpr int VEC = gated_vec<T>();
  if constexpr (ASYNC) {
    if (c < d) st_vec<T, VEC>(p, row * ld + c, ext, v);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < d) st_vec<T, 1>(p, row * ld + c + e, ext, v + e);
  }
}

// ----------------------------------------------------------------- forward
// Grid: csize * ctiles * b CTAs in clusters of csize.  SFU operations an element:
// two exponentials, a reciprocal, an inverse root (f g = w rsqrt(w (1 + e^-x)^2),
// w = 1 - a^2), two more with z; the decay's exponential is a polynomial
// (decay2), which also gives 1 - a without cancellation.
template <typename T, bool ASYNC, bool GATE, bool START>
__global__ void __launch_bounds__(kGatedThreads, 3) gated_fwd_kernel(const GatedParams p) {
  constexpr int VEC = gated_vec<T>(), E = kGatedSteps * VEC, NT = GATE ? 4 : 3;
  extern __shared__ __align__(16) char stage[];
  __shared__ float4 wsum[2][kGatedWarps][32];       // (P, Q) of the warps' steps
  __shared__ float4 csum[2][kGatedMaxCluster][32];  // (P, Q) of the cluster's tiles
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int C = p.csize, rank = (int)(blockIdx.x % (unsigned)C);
  const unsigned grp = blockIdx.x / (unsigned)C;
  const int64_t c0 = (grp % (unsigned)p.ctiles) * (int64_t)(32 * VEC), i = grp / (unsigned)p.ctiles;
  const int64_t c = c0 + lane * VEC;
  const int64_t R = p.b * p.L, nT = (p.L + kGatedChunk - 1) / kGatedChunk;
  const int iters = (int)((nT + C - 1) / C);
  char *mine = stage + warp * NT * kGatedStage;
  constexpr int kHalf = NT * kGatedWarps * kGatedStage;
  const GatedLane k = gated_lane<VEC>(p, c);
  const int64_t t_first = rank * kGatedChunk + warp * kGatedSteps;  // the warp's first step
  const int64_t row0 = i * p.L + t_first;
  const int64_t tile_rows = (int64_t)C * kGatedChunk;
  GatedSrc<T, ASYNC> su, sa, sg, sz;
  su.init(p.u, p.u_ld, row0, tile_rows, c0, lane, R, p.d);
  sa.init(p.ga, p.ga_ld, row0, tile_rows, c0, lane, R, p.d);
  sg.init(p.gx, p.gx_ld, row0, tile_rows, c0, lane, R, p.d);
  if constexpr (GATE) sz.init(p.z, p.z_ld, row0, tile_rows, c0, lane, R, p.d);
  const int piece = gated_piece<T, ASYNC>(c0, lane, p.d);
  const int64_t xy = extent(R, p.d, p.y_ld);
  float h[VEC];  // state in front of the cluster's next tiles
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = 0.0f;
    if (p.h0 && c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
      h[e] = p.h0[i * p.d + c + e];
  }
  unsigned flag = 0;  // lane r: whether a sequence starts at the next tile's row r
  // the warp's rows of its CTA's tile of round `it`
  const auto rows_of = [&](int it) {
    const int64_t left = p.L - t_first - it * tile_rows;
    return left >= kGatedSteps ? kGatedSteps : left > 0 ? (int)left : 0;
  };
  const auto fetch = [&](int it) {
    if (it < iters) {
      const int n = rows_of(it);
      char *s = mine + (it & 1) * kHalf;
      su.fetch(s, n, piece, lane);
      sa.fetch(s + kGatedStage, n, piece, lane);
      sg.fetch(s + 2 * kGatedStage, n, piece, lane);
      if constexpr (GATE) sz.fetch(s + 3 * kGatedStage, n, piece, lane);
      if (START) {
        const int64_t r = row0 + it * tile_rows + lane;
        flag = lane < n && in_bounds(r, R, kBndAct) ? p.start[r] : 0;
      }
    }
    cp_async_commit();
  };
  if (C > 1) {  // every CTA of the cluster runs before one writes to another
    cluster_arrive();
    cluster_wait();
  }
  fetch(0);
  for (int it = 0; it < iters; ++it) {
    const unsigned bits = START ? __ballot_sync(~0u, flag != 0) : 0;
    __syncwarp();  // the other half's rows are no longer read
    fetch(it + 1);
    cp_async_wait<1>();
    __syncwarp();
    const int n = rows_of(it);
    const char *s = mine + (it & 1) * kHalf;
    // decays and drives of the warp's steps, and their composition
    float a[E], x[E];
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      const float2 er = ex2_2(fma2(staged_pair<T>(s + kGatedStage, q, lane), f2(-kLog2e), k.na));
      const float2 eg = ex2_2(fma2(staged_pair<T>(s + 2 * kGatedStage, q, lane), f2(-kLog2e), k.nx));
      const float2 r = rcp_2(__fadd2_rn(er, f2(1.0f)));
      const float2 q1 = __fadd2_rn(eg, f2(1.0f));
      float2 av, w;
      decay2(mul2(k.A2, r), av, w);
      const float2 u = staged_pair<T>(s, q, lane);
      // f g = w / sqrt(w (1 + e^-x)^2)
      const float2 fg = mul2(w, rsqrt_2(mul2(mul2(w, q1), q1)));
      float2 xv = mul2(fg, u);
      if (START && bits) {
        const int s0 = 2 * q / VEC, s1 = (2 * q + 1) / VEC;
        if (bits >> s0 & 1) av.x = 0.0f, xv.x = u.x * rcp_approx(q1.x);
        if (bits >> s1 & 1) av.y = 0.0f, xv.y = u.y * rcp_approx(q1.y);
      }
      a[2 * q] = av.x, a[2 * q + 1] = av.y;
      x[2 * q] = xv.x, x[2 * q + 1] = xv.y;
    }
    if (n < kGatedSteps) {  // steps past the end change nothing
#pragma unroll
      for (int q = 0; q < E; ++q)
        if (q / VEC >= n) a[q] = 1.0f, x[q] = 0.0f;
    }
    float P[VEC], Q[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) P[e] = a[e], Q[e] = x[e];
#pragma unroll
    for (int q = VEC; q < E; ++q) {
      Q[q % VEC] = through<START>(a[q], Q[q % VEC], x[q]);
      P[q % VEC] = times<START>(P[q % VEC], a[q]);
    }
    const int par = it & 1;
    wsum[par][warp][lane] = make_float4(P[0], P[VEC - 1], Q[0], Q[VEC - 1]);
    __syncthreads();
    // composition of the steps in front of this warp's; the last warp's, with its
    // own, is the tile's
    float4 front = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
    for (int w = 0; w < warp; ++w) gated_compose<VEC, START>(front, wsum[par][w][lane]);
    if (warp == kGatedWarps - 1) {
      float4 all = front;
      gated_compose<VEC, START>(all, make_float4(P[0], P[VEC - 1], Q[0], Q[VEC - 1]));
      if (C > 1)
        for (int w = 0; w < C; ++w) st_peer(&csum[par][rank][lane], w, all);
      else
        csum[par][0][lane] = all;
    }
    gated_exchange(C, warp == kGatedWarps - 1);
    float hs[VEC];  // state in front of the warp's steps
    for (int w = 0; w < C; ++w) {
      if (w == rank) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) hs[e] = h[e];
      }
      const float4 m = csum[par][w][lane];
      h[0] = through<START>(m.x, h[0], m.z);
      if constexpr (VEC == 2) h[1] = through<START>(m.y, h[1], m.w);
    }
    const int64_t tile = it * (int64_t)C + rank;
    if (p.chunk_h && warp == 0 && tile < nT) {
      const int64_t o = (i * nT + tile) * p.d + c, on = p.b * nT * p.d;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c + e < p.d && in_bounds(o + e, on, kBndChunk)) p.chunk_h[o + e] = hs[e];
    }
    hs[0] = through<START>(front.x, hs[0], front.z);
    if constexpr (VEC == 2) hs[1] = through<START>(front.y, hs[1], front.w);
    // replay
#pragma unroll
    for (int q = 0; q < E; ++q) {
      hs[q % VEC] = through<START>(a[q], hs[q % VEC], x[q]);
      x[q] = hs[q % VEC];
    }
    if constexpr (GATE) {
#pragma unroll
      for (int q = 0; q < E / 2; ++q) {
        const float2 o = mul2(make_float2(x[2 * q], x[2 * q + 1]),
                              silu_2(staged_pair<T>(s + 3 * kGatedStage, q, lane)));
        x[2 * q] = o.x, x[2 * q + 1] = o.y;
      }
    }
    const int64_t row = row0 + it * tile_rows;
    if (n == kGatedSteps) {
#pragma unroll
      for (int t = 0; t < kGatedSteps; ++t)
        store_step<T, ASYNC>(p.y, p.y_ld, row + t, c, p.d, xy, x + t * VEC);
    } else {
#pragma unroll
      for (int t = 0; t < kGatedSteps; ++t)
        if (t < n) store_step<T, ASYNC>(p.y, p.y_ld, row + t, c, p.d, xy, x + t * VEC);
    }
  }
  if (p.h_last && rank == 0 && warp == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
        p.h_last[i * p.d + c + e] = h[e];
  }
}

// ---------------------------------------------------------------- backward
// The same tiles from the last to the first.  Per element four SFU operations (r
// and g share a reciprocal: 1 / ((1 + e^-ra)(1 + e^-gx)), exponentials capped at
// 2^60 so that their product stays finite, which bounds the gates at 2^-60 from
// below), two more with z.  a, f, a^2 / f, g and the adjoint stay in registers; r
// is put back over the staged gates it came from.
template <typename T, bool ASYNC, bool GATE, bool START>
__global__ void __launch_bounds__(kGatedThreads, 2) gated_bwd_kernel(const GatedBwdParams q_) {
  const GatedParams &p = q_.f;
  constexpr int VEC = gated_vec<T>(), E = kGatedSteps * VEC, NT = GATE ? 5 : 4;
  extern __shared__ __align__(16) char stage[];
  __shared__ float4 wsum[2][kGatedWarps][32];       // (P, mu) of the warps' steps
  __shared__ float2 wfwd[2][kGatedWarps][32];       // Q of the forward recurrence
  __shared__ float4 csum[2][kGatedMaxCluster][32];  // (P, mu) of the cluster's tiles
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int C = p.csize, rank = (int)(blockIdx.x % (unsigned)C);
  const unsigned grp = blockIdx.x / (unsigned)C;
  const int64_t c0 = (grp % (unsigned)p.ctiles) * (int64_t)(32 * VEC), i = grp / (unsigned)p.ctiles;
  const int64_t c = c0 + lane * VEC;
  const int64_t R = p.b * p.L, nT = (p.L + kGatedChunk - 1) / kGatedChunk;
  const int iters = (int)((nT + C - 1) / C);
  char *mine = stage + warp * NT * kGatedStage;
  constexpr int kHalf = NT * kGatedWarps * kGatedStage;
  const GatedLane k = gated_lane<VEC>(p, c);
  // tiles from the end: rank 0 takes the last of the cluster's
  const int64_t tile0 = nT - 1 - rank;
  const int64_t t_first = tile0 * kGatedChunk + warp * kGatedSteps;  // the warp's first step
  const int64_t row0 = i * p.L + t_first;
  const int64_t tile_rows = -(int64_t)C * kGatedChunk;
  GatedSrc<T, ASYNC> su, s_a, sg, so, sz;
  su.init(p.u, p.u_ld, row0, tile_rows, c0, lane, R, p.d);
  s_a.init(p.ga, p.ga_ld, row0, tile_rows, c0, lane, R, p.d);
  sg.init(p.gx, p.gx_ld, row0, tile_rows, c0, lane, R, p.d);
  so.init(q_.dout, q_.dout_ld, row0, tile_rows, c0, lane, R, p.d);
  if constexpr (GATE) sz.init(p.z, p.z_ld, row0, tile_rows, c0, lane, R, p.d);
  const int piece = gated_piece<T, ASYNC>(c0, lane, p.d);
  const int64_t yu = extent(R, p.d, q_.du_ld), ya = extent(R, p.d, q_.dga_ld), yg = extent(R, p.d, q_.dgx_ld),
                yz = extent(R, p.d, q_.dz_ld);
  float mu[VEC];                          // adjoint behind the cluster's next tiles
  float2 sA = f2(0.0f), sa = sA, sx = sA;  // sums of dl r, dgate_a / A, dgate_x
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    mu[e] = 0.0f;
    if (q_.dh_last && c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
      mu[e] = q_.dh_last[i * p.d + c + e];
  }
  unsigned flag = 0;
  float hnext[VEC];  // the next tile's start state
#pragma unroll
  for (int e = 0; e < VEC; ++e) hnext[e] = 0.0f;
  const auto rows_of = [&](int it) {
    if (tile0 - it * (int64_t)C < 0) return 0;
    const int64_t left = p.L - t_first - it * tile_rows;
    return left >= kGatedSteps ? kGatedSteps : left > 0 ? (int)left : 0;
  };
  const auto fetch = [&](int it) {
    if (it < iters) {
      const int n = rows_of(it);
      char *s = mine + (it & 1) * kHalf;
      su.fetch(s, n, piece, lane);
      s_a.fetch(s + kGatedStage, n, piece, lane);
      sg.fetch(s + 2 * kGatedStage, n, piece, lane);
      so.fetch(s + 3 * kGatedStage, n, piece, lane);
      if constexpr (GATE) sz.fetch(s + 4 * kGatedStage, n, piece, lane);
      if (START) {
        const int64_t r = row0 + it * tile_rows + lane;
        flag = lane < n && in_bounds(r, R, kBndAct) ? p.start[r] : 0;
      }
      const int64_t tile = tile0 - it * (int64_t)C;
      if (tile >= 0) {
        const int64_t o = (i * nT + tile) * p.d + c, on = p.b * nT * p.d;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (c + e < p.d && in_bounds(o + e, on, kBndChunk)) hnext[e] = __ldg(p.chunk_h + o + e);
      }
    }
    cp_async_commit();
  };
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  }
  fetch(0);
  for (int it = 0; it < iters; ++it) {
    const unsigned bits = START ? __ballot_sync(~0u, flag != 0) : 0;
    float hs[VEC];  // state in front of the tile, then of the warp's steps
#pragma unroll
    for (int e = 0; e < VEC; ++e) hs[e] = hnext[e];
    __syncwarp();
    fetch(it + 1);
    cp_async_wait<1>();
    __syncwarp();
    const int64_t row = row0 + it * tile_rows;
    const int n = rows_of(it);
    char *s = mine + (it & 1) * kHalf;
    float a[E], f[E], af[E], g[E], lam[E];  // af = a^2 / f; lam: dout silu(z), later the adjoint
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      float2 er = ex2_2(fma2(staged_pair<T>(s + kGatedStage, q, lane), f2(-kLog2e), k.na));
      float2 eg = ex2_2(fma2(staged_pair<T>(s + 2 * kGatedStage, q, lane), f2(-kLog2e), k.nx));
      constexpr float kCap = 1152921504606846976.0f;  // 2^60
      er = __fadd2_rn(make_float2(min_nan(er.x, kCap), min_nan(er.y, kCap)), f2(1.0f));
      eg = __fadd2_rn(make_float2(min_nan(eg.x, kCap), min_nan(eg.y, kCap)), f2(1.0f));
      const float2 inv = rcp_2(mul2(er, eg));
      const float2 r = mul2(inv, eg), gv = mul2(inv, er);
      float2 av, w;
      decay2(mul2(k.A2, r), av, w);
      float2 rho = rsqrt_2(w);
      float2 fv = mul2(w, rho);
      rho = make_float2(w.x == kDecayMinW ? 0.0f : rho.x, w.y == kDecayMinW ? 0.0f : rho.y);
      if (START && bits) {
        const int s0 = 2 * q / VEC, s1 = (2 * q + 1) / VEC;
        if (bits >> s0 & 1) av.x = 0.0f, fv.x = 1.0f, rho.x = 0.0f;
        if (bits >> s1 & 1) av.y = 0.0f, fv.y = 1.0f, rho.y = 0.0f;
      }
      const float2 afv = mul2(mul2(av, av), rho);
      float2 go = staged_pair<T>(s + 3 * kGatedStage, q, lane);
      if constexpr (GATE) go = mul2(go, silu_2(staged_pair<T>(s + 4 * kGatedStage, q, lane)));
      a[2 * q] = av.x, a[2 * q + 1] = av.y;
      f[2 * q] = fv.x, f[2 * q + 1] = fv.y;
      af[2 * q] = afv.x, af[2 * q + 1] = afv.y;
      g[2 * q] = gv.x, g[2 * q + 1] = gv.y;
      lam[2 * q] = go.x, lam[2 * q + 1] = go.y;
      // r over the gates it came from
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<float *>(s + kGatedStage + q * kGatedRowBytes + lane * 4) = r.x;
        *reinterpret_cast<float *>(s + 2 * kGatedStage + q * kGatedRowBytes + lane * 4) = r.y;
      } else {
        float *o = reinterpret_cast<float *>(s + kGatedStage) + lane;
        o[2 * q * 32] = r.x;
        o[(2 * q + 1) * 32] = r.y;
      }
    }
    if (n < kGatedSteps) {
#pragma unroll
      for (int q = 0; q < E; ++q)
        if (q / VEC >= n) a[q] = 1.0f, f[q] = 0.0f, lam[q] = 0.0f;
    }
    float P[VEC], Q[VEC], M[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) P[e] = 1.0f, Q[e] = 0.0f, M[e] = 0.0f;
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      const float2 u = staged_pair<T>(s, q, lane);
      const float2 x = mul2(mul2(make_float2(f[2 * q], f[2 * q + 1]), make_float2(g[2 * q], g[2 * q + 1])), u);
      const int e0 = (2 * q) % VEC, e1 = (2 * q + 1) % VEC;
      Q[e0] = through<START>(a[2 * q], Q[e0], x.x);
      Q[e1] = through<START>(a[2 * q + 1], Q[e1], x.y);
      P[e0] = times<START>(P[e0], a[2 * q]);
      P[e1] = times<START>(P[e1], a[2 * q + 1]);
    }
    // mu_t = a_t (go_t + mu_{t+1}); a step that starts a sequence hands nothing back
#pragma unroll
    for (int q = E - 1; q >= 0; --q) {
      const float m = a[q] * (lam[q] + M[q % VEC]);
      M[q % VEC] = START && a[q] == 0.0f ? 0.0f : m;
    }
    const int par = it & 1;
    wsum[par][warp][lane] = make_float4(P[0], P[VEC - 1], M[0], M[VEC - 1]);
    wfwd[par][warp][lane] = make_float2(Q[0], Q[VEC - 1]);
    __syncthreads();
    // the steps behind this warp's; the first warp's, with its own, is the tile's
    float4 back = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
    for (int w = kGatedWarps - 1; w > warp; --w) gated_compose<VEC, START>(back, wsum[par][w][lane]);
    if (warp == 0) {
      float4 all = back;
      gated_compose<VEC, START>(all, make_float4(P[0], P[VEC - 1], M[0], M[VEC - 1]));
      if (C > 1)
        for (int w = 0; w < C; ++w) st_peer(&csum[par][rank][lane], w, all);
      else
        csum[par][0][lane] = all;
    }
    for (int w = 0; w < warp; ++w) {
      const float4 m = wsum[par][w][lane];
      const float2 x = wfwd[par][w][lane];
      hs[0] = through<START>(m.x, hs[0], x.x);
      if constexpr (VEC == 2) hs[1] = through<START>(m.y, hs[1], x.y);
    }
    gated_exchange(C, warp == 0);
    float mb[VEC];  // adjoint behind the warp's steps
    for (int w = 0; w < C; ++w) {
      if (w == rank) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) mb[e] = mu[e];
      }
      const float4 m = csum[par][w][lane];
      mu[0] = through<START>(m.x, mu[0], m.z);
      if constexpr (VEC == 2) mu[1] = through<START>(m.y, mu[1], m.w);
    }
    mb[0] = through<START>(back.x, mb[0], back.z);
    if constexpr (VEC == 2) mb[1] = through<START>(back.y, mb[1], back.w);
    // the adjoints, last step first
#pragma unroll
    for (int q = E - 1; q >= 0; --q) {
      lam[q] += mb[q % VEC];
      const float m = a[q] * lam[q];
      mb[q % VEC] = START && a[q] == 0.0f ? 0.0f : m;
    }
    // the states, first step first, and the gradients
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      const float2 u = staged_pair<T>(s, q, lane);
      const float2 av = make_float2(a[2 * q], a[2 * q + 1]), fv = make_float2(f[2 * q], f[2 * q + 1]);
      const float2 gv = make_float2(g[2 * q], g[2 * q + 1]), lv = make_float2(lam[2 * q], lam[2 * q + 1]);
      float2 r;
      if constexpr (sizeof(T) == 2) {
        r.x = *reinterpret_cast<const float *>(s + kGatedStage + q * kGatedRowBytes + lane * 4);
        r.y = *reinterpret_cast<const float *>(s + 2 * kGatedStage + q * kGatedRowBytes + lane * 4);
      } else {
        r = staged_pair<float>(s + kGatedStage, q, lane);
      }
      const float2 gu = mul2(gv, u), x = mul2(fv, gu);
      const int e0 = (2 * q) % VEC, e1 = (2 * q + 1) % VEC;
      float2 ah, hn;  // a h_{t-1}; h_t
      ah.x = START && av.x == 0.0f ? 0.0f : av.x * hs[e0];
      hs[e0] = hn.x = ah.x + x.x;
      ah.y = START && av.y == 0.0f ? 0.0f : av.y * hs[e1];
      hs[e1] = hn.y = ah.y + x.y;
      const float2 du = mul2(mul2(lv, fv), gv);
      const float2 dgx = mul2(mul2(du, u), __ffma2_rn(gv, f2(-1.0f), f2(1.0f)));
      float2 dl = __ffma2_rn(mul2(make_float2(af[2 * q], af[2 * q + 1]), gu), f2(-1.0f), ah);
      dl = mul2(dl, lv);
      if (START) {
        if (av.x == 0.0f) dl.x = 0.0f;
        if (av.y == 0.0f) dl.y = 0.0f;
      }
      const float2 dlr = mul2(dl, r);
      float2 dga = mul2(dlr, __ffma2_rn(r, f2(-1.0f), f2(1.0f)));
      const bool on0 = (2 * q) / VEC < n, on1 = (2 * q + 1) / VEC < n;
      if (n == kGatedSteps) {
        sA = __fadd2_rn(sA, dlr);
        sa = __fadd2_rn(sa, dga);
        sx = __fadd2_rn(sx, dgx);
      } else {
        if (on0) sA.x += dlr.x, sa.x += dga.x, sx.x += dgx.x;
        if (on1) sA.y += dlr.y, sa.y += dga.y, sx.y += dgx.y;
      }
      dga = mul2(dga, mul2(k.A2, f2(kLn2)));
      const float vu[2] = {du.x, du.y}, va[2] = {dga.x, dga.y}, vg[2] = {dgx.x, dgx.y};
      float vz[2];
      if constexpr (GATE) {
        const float2 dy = staged_pair<T>(s + 3 * kGatedStage, q, lane);
        const float2 z = staged_pair<T>(s + 4 * kGatedStage, q, lane);
        const float2 sg = rcp_2(__fadd2_rn(ex2_2(mul2(z, f2(-kLog2e))), f2(1.0f)));
        // silu'(z) = s + z s (1 - s)
        const float2 ds = __ffma2_rn(mul2(z, sg), __ffma2_rn(sg, f2(-1.0f), f2(1.0f)), sg);
        const float2 dz = mul2(mul2(dy, hn), ds);
        vz[0] = dz.x, vz[1] = dz.y;
      }
#pragma unroll
      for (int e = 0; e < 2; e += VEC) {
        const int t = (2 * q + e) / VEC;
        if (t >= n) continue;
        store_step<T, ASYNC>(q_.du, q_.du_ld, row + t, c, p.d, yu, vu + e);
        store_step<T, ASYNC>(q_.dga, q_.dga_ld, row + t, c, p.d, ya, va + e);
        store_step<T, ASYNC>(q_.dgx, q_.dgx_ld, row + t, c, p.d, yg, vg + e);
        if constexpr (GATE) store_step<T, ASYNC>(q_.dz, q_.dz_ld, row + t, c, p.d, yz, vz + e);
      }
    }
  }
  if (q_.dh0 && rank == 0 && warp == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
        q_.dh0[i * p.d + c + e] = mu[e];
  }
  // the parameters' sums over the CTA's warps
  if constexpr (VEC == 1) {  // a pair holds two steps of one channel
    sA.x += sA.y, sa.x += sa.y, sx.x += sx.y;
  }
  cp_async_wait<0>();
  __syncthreads();
  float2 *red = reinterpret_cast<float2 *>(stage);  // (3, warps, 32)
  red[(0 * kGatedWarps + warp) * 32 + lane] = sA;
  red[(1 * kGatedWarps + warp) * 32 + lane] = mul2(sa, mul2(k.A2, f2(kLn2)));
  red[(2 * kGatedWarps + warp) * 32 + lane] = sx;
  __syncthreads();
  if (warp < 3) {
    float2 t = red[warp * kGatedWarps * 32 + lane];
#pragma unroll
    for (int w = 1; w < kGatedWarps; ++w) t = __fadd2_rn(t, red[(warp * kGatedWarps + w) * 32 + lane]);
    const int64_t o = ((i * C + rank) * 3 + warp) * p.d + c, on = p.b * C * 3 * p.d;
    if (c < p.d && in_bounds(o, on, kBndWork)) q_.part[o] = t.x;
    if constexpr (VEC == 2)
      if (c + 1 < p.d && in_bounds(o + 1, on, kBndWork)) q_.part[o + 1] = t.y;
  }
}

// -------------------------------------------------------------------- step
// One token, VEC channels a thread: bound by the read and write of the state and
// the activations.
template <typename T, int VEC, bool GATE>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedParams p, float *state) {
  const int64_t G = p.d / VEC;
  const int64_t k = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (k >= p.b * G) return;
  const int64_t i = p.b * G <= 0xffffffffll ? (int64_t)((unsigned)k / (unsigned)G) : k / G;
  const int64_t c = (k - i * G) * VEC, o = i * p.d + c;
  if (!in_bounds(o, p.b * p.d - (VEC - 1), kBndState)) return;
  float h[VEC], u[VEC], ga[VEC], gx[VEC], z[VEC], y[VEC];
  unpack(*reinterpret_cast<const typename VecWord<float, VEC>::type *>(state + o), h);
  unpack(ld_raw_ro<T, VEC>(p.u, i * p.u_ld + c, extent(p.b, p.d, p.u_ld)), u);
  unpack(ld_raw_ro<T, VEC>(p.ga, i * p.ga_ld + c, extent(p.b, p.d, p.ga_ld)), ga);
  unpack(ld_raw_ro<T, VEC>(p.gx, i * p.gx_ld + c, extent(p.b, p.d, p.gx_ld)), gx);
  if constexpr (GATE) unpack(ld_raw_ro<T, VEC>(p.z, i * p.z_ld + c, extent(p.b, p.d, p.z_ld)), z);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float r = sigmoid_f32(ga[e] + (p.ba ? ld_param(p.ba, c + e, p.d) : 0.0f));
    const float g = sigmoid_f32(gx[e] + (p.bx ? ld_param(p.bx, c + e, p.d) : 0.0f));
    float2 a, w;
    decay2(f2(min_nan(ld_param(p.A, c + e, p.d) * kLog2e, 126.0f) * r), a, w);
    h[e] = fmaf(a.x, h[e], w.x * rsqrt_approx(w.x) * (g * u[e]));
    y[e] = h[e];
    if constexpr (GATE) y[e] *= silu_f32(z[e]);
  }
  st_vec<float, VEC>(state, o, p.b * p.d, h);
  st_vec<T, VEC>(p.y, i * p.y_ld + c, extent(p.b, p.d, p.y_ld), y);
}

}  // namespace ssm
