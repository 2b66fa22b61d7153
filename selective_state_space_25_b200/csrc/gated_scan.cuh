// gated_scan.cuh -- the gated linear recurrence: forward, backward, one-token
// step.
//
//   r = sigmoid(ga + ba), g = sigmoid(gx + bx), a = exp(A r), f = sqrt(1 - a^2)
//   h_t = a h_{t-1} + f g u          (h_t = g u where a sequence starts)
//
// Split over time.  A step is the map h -> a h + x, and maps compose: steps
// taken together are h -> P h + Q with P the product of their decays.  A CTA's 8
// warps walk tiles of 64 S steps (bf16 backward 32 S): a lane takes VEC channels and
// 8 (4) steps, 32 / S lanes side by side the CTA's channels, the S parts of a warp and
// the warps consecutive steps.  A lane forms its decays and drives and their (P, Q) in
// registers; the parts of a warp combine by shuffles and the warps through shared
// memory; each composes what lies in front of it onto the tile's start state and
// then replays its 8 steps from registers.  So every input is read once and
// nothing waits on more than 8 sequential steps, where a thread per channel waits
// on L.  S (1, 2, 4: 128, 64, 32 bytes of a row for a CTA) trades channels for
// steps until there are CTAs enough; where that is not enough, up to 8 CTAs of a
// cluster take consecutive tiles at once and exchange the tiles' (P, Q) through
// each other's shared memory (gated_plan).
//
// The adjoint is the same recurrence backwards: mu_t = a_t (dout_t + mu_{t+1}) is
// what step t hands to step t - 1, so the backward composes (P, mu) of tiles from
// the end, and recomputes the states from those that the forward kept (4 bytes
// every 32 steps and channel).
//
// Measured (B200, b = 8, L = 2048, d = 1536, bf16, us): forward 58, backward 130
// (floors 31 and 54 at the copy bandwidth); with z 69 and 162; fp32 78 and 147 (61,
// 108).  bf16 is bound by latency at 16 warps an SM and its part-filled second wave
// (384 CTAs over 296 places): 39 and 97 instructions an element, issue slots 56-62 %
// full, SFU 47 and 28 %.
#pragma once

#include <type_traits>

#include "block_common.cuh"

namespace ssm {

struct GatedParams {
  const void *u, *ga, *gx, *z;
  int u_ld, ga_ld, gx_ld, z_ld;  // below 2^31: offsets of a few rows take one multiply
  const float *A, *ba, *bx;
  const uint8_t *start;
  const float *h0;
  float *h_last;
  void *y;
  int y_ld;
  float *chunk_h;
  int64_t b, L, d;
  int parts;    // S: parts of a warp
  int ctiles;   // CTAs across the channels
  int csize;    // CTAs of a cluster: tiles taken at once
};

struct GatedBwdParams {
  GatedParams f;  // inputs of the forward; chunk_h is read
  const void *dout;
  int dout_ld;
  const float *dh_last;
  void *du, *dga, *dgx, *dz;
  int du_ld, dga_ld, dgx_ld, dz_ld;
  float *dh0;
  float *part;  // (b * csize, 3, d): sums of dA, dbias_a, dbias_x
};

constexpr int kGatedWarps = 8;  // of a CTA
constexpr int kGatedThreads = 32 * kGatedWarps;
// Steps of a lane in a tile, and CTAs an SM holds (bf16 lanes take two channels:
// 128 registers, of which the backward spills 4 to 44 bytes in most forms).  Measured at that step (b = 8, L = 2048, d = 1536, us): bf16 forward 8
// steps with 2 CTAs 61, with 3 (spills) 64, 4 steps with 2, 3, 4 CTAs 76, 73, 79,
// 16 steps 60 (86 with z, whose stages leave room for one CTA); backward 4 steps
// with 2 CTAs 145, with 3 (spills) 179, 8 steps with 2 (spills) 178, with 1 168.
// fp32 forward with 2, 3 CTAs 86, 78; backward 4 steps with 3 CTAs 201, 8 with 2 145.
constexpr int kGatedFwdSteps = 8;
template <typename T> constexpr int gated_bwd_steps() { return sizeof(T) == 2 ? 4 : 8; }
template <typename T> constexpr int gated_ctas() { return sizeof(T) == 2 ? 2 : 3; }
constexpr int kGatedBwdCtas = 2;
static_assert(kGatedChunk % (4 * kGatedFwdSteps) == 0, "a chunk is whole warps, whatever S");
constexpr int kGatedMaxCluster = 8;
constexpr int kGatedRowBytes = 128;

// Channels a lane takes: 32 VEC channels are 128 bytes.
template <typename T> constexpr int gated_vec() { return 4 / (int)sizeof(T); }

// Dynamic shared memory of a CTA: NT tensors' rows of two tiles, then the
// compositions of the cluster's tiles, for two rounds.
constexpr int gated_stage(int nt, int steps) { return nt * kGatedWarps * steps * kGatedRowBytes; }
constexpr int kGatedStages = 2;
constexpr int gated_smem(int nt, int steps, int csize) {
  return kGatedStages * gated_stage(nt, steps) + 2 * csize * 32 * 16;
}

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
// Only a start makes P 0: a step's decay is at least 2^-126 (decay2), and a product
// of decays is held at the smallest fp32 number, where it would round to 0.  So a
// NaN or an infinite state stays one until a sequence starts (fma(0, inf, Q) would
// be NaN, too), and a finite one is off by 2^-149 of itself at most.
constexpr float kDecayMinP = 1.40129846e-45f;  // 2^-149
template <bool START> __device__ __forceinline__ float through(float P, float h, float Q) {
  const float r = fmaf(P, h, Q);
  return START && P == 0.0f ? Q : r;
}
// Product of two maps' decays; with START one of 0 stays 0 beside a NaN.
template <bool START> __device__ __forceinline__ float times(float P, float a) {
  if constexpr (!START) return P * a;  // held above 0 where its composition ends
  const float r = max_nan(P * a, kDecayMinP);
  return P == 0.0f || a == 0.0f ? 0.0f : r;
}

// States of VEC channels after the map m, (P, P, Q, Q).
template <int VEC, bool START> __device__ __forceinline__ void gated_apply(float (&h)[VEC], float4 m) {
  if constexpr (VEC == 2 && !START) {
    const float2 r = __ffma2_rn(make_float2(m.x, m.y), make_float2(h[0], h[1]), make_float2(m.z, m.w));
    h[0] = r.x, h[1] = r.y;
  } else {
    h[0] = through<START>(m.x, h[0], m.z);
    if constexpr (VEC == 2) h[1] = through<START>(m.y, h[1], m.w);
  }
}
// Flat elements 2 q and 2 q + 1 of a lane (one step of two channels, or two steps
// of one) taken into the state h, and into the product P of the decays.
template <int VEC, bool START>
__device__ __forceinline__ void gated_step2(float (&h)[VEC], const float *a, const float *x) {
  if constexpr (VEC == 2) {
    gated_apply<2, START>(h, make_float4(a[0], a[1], x[0], x[1]));
  } else {
    h[0] = through<START>(a[0], h[0], x[0]);
    h[0] = through<START>(a[1], h[0], x[1]);
  }
}
template <int VEC> __device__ __forceinline__ void gated_prod2(float (&P)[VEC], const float *a) {
  if constexpr (VEC == 2) {
    const float2 r = __fmul2_rn(make_float2(P[0], P[1]), make_float2(a[0], a[1]));
    P[0] = r.x, P[1] = r.y;
  } else {
    P[0] = P[0] * a[0] * a[1];
  }
}
// The product of a lane's steps as a map's: 0 where a sequence starts among them.
template <int VEC> __device__ __forceinline__ void gated_prod_end(float (&P)[VEC], bool start) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) P[e] = start ? 0.0f : max_nan(P[e], kDecayMinP);
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

// Ends a composition: its P as other maps and states meet it.
template <int VEC, bool START> __device__ __forceinline__ void gated_compose_end(float4 &m) {
  if constexpr (!START) {
    m.x = max_nan(m.x, kDecayMinP);
    if constexpr (VEC == 2) m.y = max_nan(m.y, kDecayMinP);
  }
}

// (P, P, Q, Q) of another lane.
__device__ __forceinline__ float4 shfl4(float4 v, int lane) {
  return make_float4(__shfl_sync(~0u, v.x, lane), __shfl_sync(~0u, v.y, lane),
                     __shfl_sync(~0u, v.z, lane), __shfl_sync(~0u, v.w, lane));
}

// The parts of a warp in the order they are taken (FORWARD: part 0 first, else the
// last part first): own becomes the composition of the parts taken before this
// lane's (not to be used by the part taken first), all, in the lanes of the part
// taken last, that of the warp's.
template <int VEC, bool START, bool FORWARD>
__device__ __forceinline__ void gated_parts(int S, int lane, float4 &own, float4 &all) {
  all = own;
  if (S == 1) return;
  const float4 mine = own;
  if (S == 2) {
    own = shfl4(mine, lane ^ 16);
    all = own;
    gated_compose<VEC, START>(all, mine);
    gated_compose_end<VEC, START>(all);
    return;
  }
  const int lc = 32 / S, part = lane / lc, l = lane % lc;
  all = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
  for (int k = 0; k < S; ++k) {
    const int s = FORWARD ? k : S - 1 - k;
    const float4 m = shfl4(mine, s * lc + l);
    if (s == part) own = all;
    gated_compose<VEC, START>(all, m);
  }
  gated_compose_end<VEC, START>(own);
  gated_compose_end<VEC, START>(all);
}

// Makes the tiles' compositions, which one warp of each CTA wrote, known to all
// of the cluster.  Only that warp releases at cluster scope (a release waits for
// a warp's global stores too): its release covers what the CTA's other warps
// read of the buffer two rounds ago, which the round's __syncthreads ordered
// before it.
__device__ __forceinline__ void gated_arrive(bool writer) {
  __syncwarp();
  if (writer)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
  l.na = mul2(lane_pair<VEC>(p.ba, c, p.d), f2(-kLog2e));
  l.nx = mul2(lane_pair<VEC>(p.bx, c, p.d), f2(-kLog2e));
  return l;
}

// ----------------------------------------------------------------- staging
// One tensor's rows for a warp, `step` bytes to the next tile's.  In shared memory
// step k of all parts lies side by side, 128 bytes, lane l's channels at 4 l (so
// that a warp reads each bank once).  ASYNC: 16-byte cp.async (rows 16-byte
// aligned, d a multiple of 16 bytes), lane l the 16 bytes l % 8 of steps l / 8 (and
// l / 8 + 4); else element loads.  Rows past the end and channels past d become zeros.
template <typename T, bool ASYNC, int STEPS> struct GatedSrc {
  const char *p;        // the lane's first element of the next tile
  const char *lo, *hi;  // the buffer (past-the-end pieces, debug-bounds build)
  // row: the warp's first
  __device__ __forceinline__ void init(const void *src, int ld, int64_t row, int64_t c0, int lane,
                                       int64_t rows, int64_t d, int S) {
    lo = static_cast<const char *>(src);
    hi = lo + extent(rows, d, ld) * (int64_t)sizeof(T);
    const int lc = 32 / S, pc = 8 / S;  // lanes, 16-byte pieces of a part
    const int64_t r = row + (ASYNC ? lane % 8 / pc * STEPS + lane / 8 : lane / lc * STEPS);
    p = lo + (r * ld + c0) * (int64_t)sizeof(T) +
        (ASYNC ? lane % 8 % pc * 16 : lane % lc * gated_vec<T>() * (int)sizeof(T));
  }
  // n rows of this tile for the part whose bytes the lane copies; bytes: 16 where
  // its piece lies in front of d, else 0 (elements: how many of the lane's do);
  // then on by tile_rows rows
  __device__ __forceinline__ void fetch(char *s, int n, int bytes, int lane, int ld, int tile_rows) {
    if constexpr (ASYNC) {
#pragma unroll
      for (int j = 0; j < STEPS / 4; ++j) {
        const char *q = p + (int64_t)ld * (4 * j * (int)sizeof(T));
        int b = bytes;
        if (n < STEPS && lane / 8 + 4 * j >= n) b = 0;
        if (b && !in_bounds(q - lo, hi - lo - 15, kBndAct)) b = 0;
        if (n < STEPS && !b) q = lo;
        cp_async16(s + j * 512 + lane * 16, q, b);
      }
    } else {
      constexpr int VEC = gated_vec<T>();
      T v[STEPS][VEC];
#pragma unroll
      for (int r = 0; r < STEPS; ++r)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const char *q = p + (int64_t)ld * (r * (int)sizeof(T)) + e * (int)sizeof(T);
          v[r][e] = r < n && e < bytes && in_bounds(q - lo, hi - lo, kBndAct)
                        ? *reinterpret_cast<const T *>(q) : T(0.0f);
        }
#pragma unroll
      for (int r = 0; r < STEPS; ++r)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          reinterpret_cast<T *>(s + r * kGatedRowBytes)[lane * VEC + e] = v[r][e];
    }
    p += (int64_t)ld * (tile_rows * (int)sizeof(T));
  }
};
// The `bytes` of fetch for a lane.
template <typename T, bool ASYNC>
__device__ __forceinline__ int gated_piece(int64_t c0, int lane, int64_t d, int S) {
  if constexpr (ASYNC) return c0 + lane % 8 % (8 / S) * (16 / (int)sizeof(T)) < d ? 16 : 0;
  const int64_t left = d - c0 - lane % (32 / S) * gated_vec<T>();
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

// An output's place: the lane's channels in the first of its steps of a tile.
template <typename T, bool ASYNC> struct GatedDst {
  T *p, *lo;
  int64_t n;  // elements of the buffer (debug-bounds build)
  __device__ __forceinline__ void init(void *dst, int ld, int64_t row, int64_t c, int64_t rows, int64_t d) {
    lo = static_cast<T *>(dst);
    n = extent(rows, d, ld);
    p = lo + (row * ld + c);
  }
  // VEC channels of step t of the tile, `left` of them in front of d
  __device__ __forceinline__ void store(int t, int ld, int left, const float *v) const {
    constexpr int VEC = gated_vec<T>();
    T *q = p + (int64_t)ld * t;
    if constexpr (ASYNC) {
      if (left > 0 && in_bounds(q - lo, n - (VEC - 1), kBndAct)) st_vec<T, VEC>(q, 0, VEC, v);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < left && in_bounds(q + e - lo, n, kBndAct)) st_vec<T, 1>(q, e, VEC, v + e);
    }
  }
  __device__ __forceinline__ void next(int ld, int tile_rows) { p += (int64_t)ld * tile_rows; }
};

// ----------------------------------------------------------------- forward
// Grid: csize * ctiles * b CTAs in clusters of csize.  SFU operations an element:
// two exponentials, a reciprocal, an inverse root (f g = w rsqrt(w (1 + e^-x)^2),
// w = 1 - a^2), two more with z; the decay's exponential is a polynomial
// (decay2), which also gives 1 - a without cancellation.  Where g is below some
// 2^-64, w (1 + e^-x)^2 is infinite and the drive 0.
template <typename T, bool ASYNC, bool GATE, bool START>
__global__ void __launch_bounds__(kGatedThreads, gated_ctas<T>()) gated_fwd_kernel(const GatedParams p) {
  constexpr int STEPS = kGatedFwdSteps, VEC = gated_vec<T>(), E = STEPS * VEC, NT = GATE ? 4 : 3;
  constexpr int kRows = STEPS * kGatedRowBytes;  // bytes of a tensor's rows for a warp
  extern __shared__ __align__(16) char stage[];
  __shared__ float4 wsum[2][kGatedWarps][32];       // (P, Q) of the warps' steps
  float4 *const csum =
      reinterpret_cast<float4 *>(stage + kGatedStages * gated_stage(NT, STEPS));  // [2][C][32]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int C = p.csize, rank = (int)(blockIdx.x % (unsigned)C);
  const unsigned grp = blockIdx.x / (unsigned)C;
  const int S = p.parts, lc = 32 / S, part = lane / lc;
  const int64_t c0 = (grp % (unsigned)p.ctiles) * (int64_t)(lc * VEC), i = grp / (unsigned)p.ctiles;
  const int64_t c = c0 + lane % lc * VEC;
  const int64_t R = p.b * p.L;
  const int L = (int)p.L, tile_rows = C * S * kGatedWarps * STEPS;  // of the cluster
  const int iters = (L + tile_rows - 1) / tile_rows;
  char *mine = stage + warp * NT * kRows;
  constexpr int kHalf = gated_stage(NT, STEPS);
  const GatedLane k = gated_lane<VEC>(p, c);
  // the warp's first step, the lane's, and that of the part it copies for
  const int t_warp = (rank * kGatedWarps + warp) * (S * STEPS);
  const int t_lane = t_warp + part * STEPS;
  const int t_copy = ASYNC ? t_warp + lane % 8 / (8 / S) * STEPS : t_lane;
  GatedSrc<T, ASYNC, STEPS> su, sa, sg, sz;
  su.init(p.u, p.u_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  sa.init(p.ga, p.ga_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  sg.init(p.gx, p.gx_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  if constexpr (GATE) sz.init(p.z, p.z_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  const int piece = gated_piece<T, ASYNC>(c0, lane, p.d, S);
  GatedDst<T, ASYNC> dy;
  dy.init(p.y, p.y_ld, i * p.L + t_lane, c, R, p.d);
  const int left = (int)(p.d - c < VEC ? p.d - c : VEC);  // channels in front of d
  float h[VEC];  // state in front of the cluster's next tiles
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    h[e] = 0.0f;
    if (p.h0 && c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
      h[e] = p.h0[i * p.d + c + e];
  }
  unsigned flag = 0;  // lane r: whether a sequence starts at the warp's next row r
  // rows from step t on of round `it`
  const auto rows_of = [&](int t, int it) {
    const int left = L - t - it * tile_rows;
    return left >= STEPS ? STEPS : left > 0 ? left : 0;
  };
  const auto fetch = [&](int it) {
    if (it < iters) {
      const int n = rows_of(t_copy, it);
      char *s = mine + (it & 1) * kHalf;
      su.fetch(s, n, piece, lane, p.u_ld, tile_rows);
      sa.fetch(s + kRows, n, piece, lane, p.ga_ld, tile_rows);
      sg.fetch(s + 2 * kRows, n, piece, lane, p.gx_ld, tile_rows);
      if constexpr (GATE) sz.fetch(s + 3 * kRows, n, piece, lane, p.z_ld, tile_rows);
      if (START) {
        const int t = t_warp + it * tile_rows + lane;
        const int64_t r = i * p.L + t;
        flag = lane < S * STEPS && t < L && in_bounds(r, R, kBndAct) ? p.start[r] : 0;
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
    const unsigned bits = START ? __ballot_sync(~0u, flag != 0) >> (part * STEPS) & ((1u << STEPS) - 1) : 0;
    const bool any = START && __any_sync(~0u, bits != 0);
    __syncwarp();  // the other half's rows are no longer read
    fetch(it + 1);
    cp_async_wait<1>();
    __syncwarp();
    const int n = rows_of(t_lane, it);
    const char *s = mine + (it & 1) * kHalf;
    // decays and drives of the warp's steps, and their composition
    float a[E], x[E];
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      const float2 er = ex2_2(fma2(staged_pair<T>(s + kRows, q, lane), f2(-kLog2e), k.na));
      const float2 eg = ex2_2(fma2(staged_pair<T>(s + 2 * kRows, q, lane), f2(-kLog2e), k.nx));
      const float2 r = rcp_2(__fadd2_rn(er, f2(1.0f)));
      const float2 q1 = __fadd2_rn(eg, f2(1.0f));
      float2 av, w;
      decay2(mul2(k.A2, r), av, w);
      const float2 u = staged_pair<T>(s, q, lane);
      // f g = w / sqrt(w (1 + e^-x)^2)
      const float2 fg = mul2(w, rsqrt_2(mul2(mul2(w, q1), q1)));
      float2 xv = mul2(fg, u);
      if (START && any) {
        const int s0 = 2 * q / VEC, s1 = (2 * q + 1) / VEC;
        if (bits >> s0 & 1) av.x = 0.0f, xv.x = u.x * rcp_approx(q1.x);
        if (bits >> s1 & 1) av.y = 0.0f, xv.y = u.y * rcp_approx(q1.y);
      }
      a[2 * q] = av.x, a[2 * q + 1] = av.y;
      x[2 * q] = xv.x, x[2 * q + 1] = xv.y;
    }
    if (n < STEPS) {  // steps past the end change nothing
#pragma unroll
      for (int q = 0; q < E; ++q)
        if (q / VEC >= n) a[q] = 1.0f, x[q] = 0.0f;
    }
    float P[VEC], Q[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) P[e] = 1.0f, Q[e] = 0.0f;
    // (only where a sequence starts among the warp's steps do they need its care)
    if (START && any) {
#pragma unroll
      for (int q = 0; q < E; q += 2) {
        gated_step2<VEC, true>(Q, a + q, x + q);
        gated_prod2<VEC>(P, a + q);
      }
    } else {
#pragma unroll
      for (int q = 0; q < E; q += 2) {
        gated_step2<VEC, false>(Q, a + q, x + q);
        gated_prod2<VEC>(P, a + q);
      }
    }
    gated_prod_end<VEC>(P, START && bits != 0);
    const int par = it & 1;
    float4 front = make_float4(P[0], P[VEC - 1], Q[0], Q[VEC - 1]), own_warp;
    gated_parts<VEC, START, true>(S, lane, front, own_warp);  // in the warp
    const int l = lane % lc;
    if (part == S - 1) wsum[par][warp][l] = own_warp;
    __syncthreads();
    float hs[VEC];  // state in front of the warp's steps
    if (C == 1) {  // the warps' maps in order from the tile's start state
#pragma unroll
      for (int e = 0; e < VEC; ++e) hs[e] = h[e];
#pragma unroll
      for (int w = 0; w < kGatedWarps; ++w) {
        gated_apply<VEC, START>(h, wsum[par][w][l]);
        if (w + 1 == warp) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) hs[e] = h[e];
        }
      }
    } else {
      // composition of the warps in front of this one; the last warp's, with its
      // own, is the tile's
      float4 ahead = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
      for (int w = 0; w < warp; ++w) gated_compose<VEC, START>(ahead, wsum[par][w][l]);
      if (warp == kGatedWarps - 1) {
        float4 all = ahead;
        gated_compose<VEC, START>(all, wsum[par][warp][l]);
        gated_compose_end<VEC, START>(all);
        for (int w = 0; w < C; ++w) st_peer(&csum[(par * C + rank) * 32 + lane], w, all);
      }
      gated_arrive(warp == kGatedWarps - 1);
      cluster_wait();
      for (int w = 0; w < C; ++w) {
        if (w == rank) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) hs[e] = h[e];
        }
        gated_apply<VEC, START>(h, csum[(par * C + w) * 32 + lane]);
      }
      gated_compose_end<VEC, START>(ahead);
      gated_apply<VEC, START>(hs, ahead);
    }
    const int t_now = t_warp + it * tile_rows;
    if (p.chunk_h && t_now % kGatedChunk == 0 && t_now < L && part == 0) {
      const int64_t nC = (L + kGatedChunk - 1) / kGatedChunk;
      const int64_t o = (i * nC + t_now / kGatedChunk) * p.d + c, on = p.b * nC * p.d;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c + e < p.d && in_bounds(o + e, on, kBndChunk)) p.chunk_h[o + e] = hs[e];
    }
    if (part > 0) gated_apply<VEC, START>(hs, front);
    // replay
    const auto replay = [&](auto care) {
      constexpr bool CARE = decltype(care)::value;
#pragma unroll
      for (int q = 0; q < E; q += VEC) {
        if constexpr (VEC == 2)
          gated_step2<VEC, CARE>(hs, a + q, x + q);
        else
          hs[0] = through<CARE>(a[q], hs[0], x[q]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[q + e] = hs[e];
      }
    };
    if (START && any)
      replay(std::true_type());
    else
      replay(std::false_type());
    if constexpr (GATE) {
#pragma unroll
      for (int q = 0; q < E / 2; ++q) {
        const float2 o = mul2(make_float2(x[2 * q], x[2 * q + 1]),
                              silu_2(staged_pair<T>(s + 3 * kRows, q, lane)));
        x[2 * q] = o.x, x[2 * q + 1] = o.y;
      }
    }
    if (n == STEPS) {
#pragma unroll
      for (int t = 0; t < STEPS; ++t) dy.store(t, p.y_ld, left, x + t * VEC);
    } else {
#pragma unroll
      for (int t = 0; t < STEPS; ++t)
        if (t < n) dy.store(t, p.y_ld, left, x + t * VEC);
    }
    dy.next(p.y_ld, tile_rows);
  }
  if (p.h_last && rank == 0 && warp == 0 && part == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
        p.h_last[i * p.d + c + e] = h[e];
  }
}

// ---------------------------------------------------------------- backward
// The same tiles from the last to the first.  Per element five SFU operations, two
// more with z.  a, f, a^2 / f, g and the adjoint stay in registers; r
// is put back over the staged gates it came from.
template <typename T, bool ASYNC, bool GATE, bool START>
__global__ void __launch_bounds__(kGatedThreads, kGatedBwdCtas) gated_bwd_kernel(const GatedBwdParams q_) {
  const GatedParams &p = q_.f;
  constexpr int STEPS = gated_bwd_steps<T>(), VEC = gated_vec<T>(), E = STEPS * VEC, NT = GATE ? 5 : 4;
  constexpr int kRows = STEPS * kGatedRowBytes;  // bytes of a tensor's rows for a warp
  extern __shared__ __align__(16) char stage[];
  __shared__ float4 wsum[2][kGatedWarps][32];       // (P, mu) of the warps' steps
  __shared__ float2 wfwd[2][kGatedWarps][32];       // Q of the forward recurrence
  float4 *const csum =
      reinterpret_cast<float4 *>(stage + kGatedStages * gated_stage(NT, STEPS));  // [2][C][32]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int C = p.csize, rank = (int)(blockIdx.x % (unsigned)C);
  const unsigned grp = blockIdx.x / (unsigned)C;
  const int S = p.parts, lc = 32 / S, part = lane / lc;
  const int64_t c0 = (grp % (unsigned)p.ctiles) * (int64_t)(lc * VEC), i = grp / (unsigned)p.ctiles;
  const int64_t c = c0 + lane % lc * VEC;
  const int64_t R = p.b * p.L;
  const int L = (int)p.L, own_rows = S * kGatedWarps * STEPS;  // of a tile
  const int nT = (L + own_rows - 1) / own_rows;
  const int iters = (nT + C - 1) / C;
  char *mine = stage + warp * NT * kRows;
  constexpr int kHalf = gated_stage(NT, STEPS);
  const GatedLane k = gated_lane<VEC>(p, c);
  // tiles from the end: rank 0 takes the last of the cluster's
  const int tile0 = nT - 1 - rank;
  const int tile_rows = -C * own_rows;
  // the warp's first step, the lane's, and that of the part it copies for
  const int t_warp = tile0 * own_rows + warp * (S * STEPS);
  const int t_lane = t_warp + part * STEPS;
  const int t_copy = ASYNC ? t_warp + lane % 8 / (8 / S) * STEPS : t_lane;
  GatedSrc<T, ASYNC, STEPS> su, s_a, sg, so, sz;
  su.init(p.u, p.u_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  s_a.init(p.ga, p.ga_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  sg.init(p.gx, p.gx_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  so.init(q_.dout, q_.dout_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  if constexpr (GATE) sz.init(p.z, p.z_ld, i * p.L + t_warp, c0, lane, R, p.d, S);
  const int piece = gated_piece<T, ASYNC>(c0, lane, p.d, S);
  GatedDst<T, ASYNC> du_, da_, dg_, dz_;
  du_.init(q_.du, q_.du_ld, i * p.L + t_lane, c, R, p.d);
  da_.init(q_.dga, q_.dga_ld, i * p.L + t_lane, c, R, p.d);
  dg_.init(q_.dgx, q_.dgx_ld, i * p.L + t_lane, c, R, p.d);
  if constexpr (GATE) dz_.init(q_.dz, q_.dz_ld, i * p.L + t_lane, c, R, p.d);
  const int left = (int)(p.d - c < VEC ? p.d - c : VEC);  // channels in front of d
  float mu[VEC];                          // adjoint behind the cluster's next tiles
  float2 sA = f2(0.0f), sa = sA, sx = sA;  // sums of dl r, dgate_a / A, dgate_x
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    mu[e] = 0.0f;
    if (q_.dh_last && c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
      mu[e] = q_.dh_last[i * p.d + c + e];
  }
  unsigned flag = 0;
  const int64_t nC = (L + kGatedChunk - 1) / kGatedChunk;
  const float *chunk = p.chunk_h + ((i * nC + (int64_t)(t_warp / kGatedChunk)) * p.d + c);
  const int64_t chunk_step = (int64_t)(tile_rows / kGatedChunk) * p.d;
  float hnext[VEC];  // state in front of the warp's next chunk
#pragma unroll
  for (int e = 0; e < VEC; ++e) hnext[e] = 0.0f;
  const auto rows_of = [&](int t, int it) {
    if (tile0 - it * C < 0) return 0;
    const int left = L - t - it * tile_rows;
    return left >= STEPS ? STEPS : left > 0 ? left : 0;
  };
  const auto fetch = [&](int it) {
    if (it < iters) {
      const int n = rows_of(t_copy, it);
      char *s = mine + (it & 1) * kHalf;
      su.fetch(s, n, piece, lane, p.u_ld, tile_rows);
      s_a.fetch(s + kRows, n, piece, lane, p.ga_ld, tile_rows);
      sg.fetch(s + 2 * kRows, n, piece, lane, p.gx_ld, tile_rows);
      so.fetch(s + 3 * kRows, n, piece, lane, q_.dout_ld, tile_rows);
      if constexpr (GATE) sz.fetch(s + 4 * kRows, n, piece, lane, p.z_ld, tile_rows);
      if (START) {
        const int t = t_warp + it * tile_rows + lane;
        const int64_t r = i * p.L + t;
        flag = lane < S * STEPS && t >= 0 && t < L && in_bounds(r, R, kBndAct) ? p.start[r] : 0;
      }
      const int t_now = t_warp + it * tile_rows;
      if (t_now >= 0 && t_now < L) {  // state in front of the warp's chunk
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e < left && in_bounds(chunk + e - p.chunk_h, p.b * nC * p.d, kBndChunk))
            hnext[e] = __ldg(chunk + e);
      }
      chunk += chunk_step;
    }
    cp_async_commit();
  };
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  }
  fetch(0);
  for (int it = 0; it < iters; ++it) {
    const unsigned bits = START ? __ballot_sync(~0u, flag != 0) >> (part * STEPS) & ((1u << STEPS) - 1) : 0;
    const bool any = START && __any_sync(~0u, bits != 0);
    float hs[VEC];  // state in front of the chunk, then of the lane's steps
#pragma unroll
    for (int e = 0; e < VEC; ++e) hs[e] = hnext[e];
    __syncwarp();
    fetch(it + 1);
    cp_async_wait<1>();
    __syncwarp();
    const int n = rows_of(t_lane, it);
    char *s = mine + (it & 1) * kHalf;
    float a[E], f[E], af[E], g[E], lam[E];  // af = a^2 / f; lam: dout silu(z), later the adjoint
#pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      const float2 er = ex2_2(fma2(staged_pair<T>(s + kRows, q, lane), f2(-kLog2e), k.na));
      const float2 eg = ex2_2(fma2(staged_pair<T>(s + 2 * kRows, q, lane), f2(-kLog2e), k.nx));
      const float2 r = rcp_2(__fadd2_rn(er, f2(1.0f))), gv = rcp_2(__fadd2_rn(eg, f2(1.0f)));
      float2 av, w;
      decay2(mul2(k.A2, r), av, w);
      float2 rho = rsqrt_2(w);
      float2 fv = mul2(w, rho);
      rho = make_float2(w.x == kDecayMinW ? 0.0f : rho.x, w.y == kDecayMinW ? 0.0f : rho.y);
      if (START && any) {
        const int s0 = 2 * q / VEC, s1 = (2 * q + 1) / VEC;
        if (bits >> s0 & 1) av.x = 0.0f, fv.x = 1.0f, rho.x = 0.0f;
        if (bits >> s1 & 1) av.y = 0.0f, fv.y = 1.0f, rho.y = 0.0f;
      }
      const float2 afv = mul2(mul2(av, av), rho);
      float2 go = staged_pair<T>(s + 3 * kRows, q, lane);
      if constexpr (GATE) go = mul2(go, silu_2(staged_pair<T>(s + 4 * kRows, q, lane)));
      a[2 * q] = av.x, a[2 * q + 1] = av.y;
      f[2 * q] = fv.x, f[2 * q + 1] = fv.y;
      af[2 * q] = afv.x, af[2 * q + 1] = afv.y;
      g[2 * q] = gv.x, g[2 * q + 1] = gv.y;
      lam[2 * q] = go.x, lam[2 * q + 1] = go.y;
      // r over the gates it came from
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<float *>(s + kRows + q * kGatedRowBytes + lane * 4) = r.x;
        *reinterpret_cast<float *>(s + 2 * kRows + q * kGatedRowBytes + lane * 4) = r.y;
      } else {
        float *o = reinterpret_cast<float *>(s + kRows) + lane;
        o[2 * q * 32] = r.x;
        o[(2 * q + 1) * 32] = r.y;
      }
    }
    if (n < STEPS) {
#pragma unroll
      for (int q = 0; q < E; ++q)
        if (q / VEC >= n) a[q] = 1.0f, f[q] = 0.0f, lam[q] = 0.0f;
    }
    float P[VEC], Q[VEC], M[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) P[e] = 1.0f, Q[e] = 0.0f, M[e] = 0.0f;
    const auto compose = [&](auto care) {  // care: a sequence starts among the warp's steps
      constexpr bool CARE = decltype(care)::value;
#pragma unroll
      for (int q = 0; q < E / 2; ++q) {
        const float2 u = staged_pair<T>(s, q, lane);
        const float2 x =
            mul2(mul2(make_float2(f[2 * q], f[2 * q + 1]), make_float2(g[2 * q], g[2 * q + 1])), u);
        const float xv[2] = {x.x, x.y};
        gated_step2<VEC, CARE>(Q, a + 2 * q, xv);
        gated_prod2<VEC>(P, a + 2 * q);
      }
      gated_prod_end<VEC>(P, CARE && bits != 0);
      // mu_t = a_t (go_t + mu_{t+1}); a step that starts a sequence hands nothing back
#pragma unroll
      for (int q = E - 1; q >= 0; --q) {
        const float m = a[q] * (lam[q] + M[q % VEC]);
        M[q % VEC] = CARE && a[q] == 0.0f ? 0.0f : m;
      }
    };
    if (START && any)
      compose(std::true_type());
    else
      compose(std::false_type());
    const int par = it & 1;
    // in the warp: back, what lies behind the lane's steps; ahead, in front of them
    float4 back = make_float4(P[0], P[VEC - 1], M[0], M[VEC - 1]), own_warp;
    float4 ahead = make_float4(P[0], P[VEC - 1], Q[0], Q[VEC - 1]), fwd_warp;
    gated_parts<VEC, START, false>(S, lane, back, own_warp);
    gated_parts<VEC, START, true>(S, lane, ahead, fwd_warp);
    const int l = lane % lc;
    if (part == 0) wsum[par][warp][l] = own_warp;
    if (part == S - 1) wfwd[par][warp][l] = make_float2(fwd_warp.z, fwd_warp.w);
    __syncthreads();
    // from the chunk's start state, through its warps in front of this one
    const int first = warp - warp % (kGatedChunk / STEPS / S);  // of the chunk
    for (int w = first; w < warp; ++w) {
      const float4 m = wsum[par][w][l];
      const float2 x = wfwd[par][w][l];
      gated_apply<VEC, START>(hs, make_float4(m.x, m.y, x.x, x.y));
    }
    if (part > 0) gated_apply<VEC, START>(hs, ahead);
    float mb[VEC];  // adjoint behind the warp's steps
    if (C == 1) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) mb[e] = mu[e];
#pragma unroll
      for (int w = kGatedWarps - 1; w >= 0; --w) {
        gated_apply<VEC, START>(mu, wsum[par][w][l]);
        if (w - 1 == warp) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) mb[e] = mu[e];
        }
      }
    } else {
      // the warps behind this one; the first warp's, with its own, is the tile's
      float4 behind = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
      for (int w = kGatedWarps - 1; w > warp; --w) gated_compose<VEC, START>(behind, wsum[par][w][l]);
      if (warp == 0) {
        float4 all = behind;
        gated_compose<VEC, START>(all, wsum[par][warp][l]);
        gated_compose_end<VEC, START>(all);
        for (int w = 0; w < C; ++w) st_peer(&csum[(par * C + rank) * 32 + lane], w, all);
      }
      gated_arrive(warp == 0);
      cluster_wait();
      for (int w = 0; w < C; ++w) {
        if (w == rank) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) mb[e] = mu[e];
        }
        gated_apply<VEC, START>(mu, csum[(par * C + w) * 32 + lane]);
      }
      gated_compose_end<VEC, START>(behind);
      gated_apply<VEC, START>(mb, behind);
    }
    if (part < S - 1) gated_apply<VEC, START>(mb, back);
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
        r.x = *reinterpret_cast<const float *>(s + kRows + q * kGatedRowBytes + lane * 4);
        r.y = *reinterpret_cast<const float *>(s + 2 * kRows + q * kGatedRowBytes + lane * 4);
      } else {
        r = staged_pair<float>(s + kRows, q, lane);
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
      if (n == STEPS) {
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
        const float2 dy = staged_pair<T>(s + 3 * kRows, q, lane);
        const float2 z = staged_pair<T>(s + 4 * kRows, q, lane);
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
        du_.store(t, q_.du_ld, left, vu + e);
        da_.store(t, q_.dga_ld, left, va + e);
        dg_.store(t, q_.dgx_ld, left, vg + e);
        if constexpr (GATE) dz_.store(t, q_.dz_ld, left, vz + e);
      }
    }
    du_.next(q_.du_ld, tile_rows);
    da_.next(q_.dga_ld, tile_rows);
    dg_.next(q_.dgx_ld, tile_rows);
    if constexpr (GATE) dz_.next(q_.dz_ld, tile_rows);
  }
  if (q_.dh0 && rank == 0 && warp == 0 && part == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < p.d && in_bounds(i * p.d + c + e, p.b * p.d, kBndState))
        q_.dh0[i * p.d + c + e] = mu[e];
  }
  // the parameters' sums over the CTA's warps and their parts
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
  if (warp < 3 && part == 0) {
    float2 t = f2(0.0f);
    for (int w = 0; w < kGatedWarps; ++w)
      for (int s = 0; s < S; ++s) t = __fadd2_rn(t, red[(warp * kGatedWarps + w) * 32 + s * lc + lane]);
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
    decay2(f2(ld_param(p.A, c + e, p.d) * kLog2e * r), a, w);
    h[e] = fmaf(a.x, h[e], w.x * rsqrt_approx(w.x) * (g * u[e]));
    y[e] = h[e];
    if constexpr (GATE) y[e] *= silu_f32(z[e]);
  }
  st_vec<float, VEC>(state, o, p.b * p.d, h);
  st_vec<T, VEC>(p.y, i * p.y_ld + c, extent(p.b, p.d, p.y_ld), y);
}

}  // namespace ssm
