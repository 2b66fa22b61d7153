// conv1d.cuh -- the causal depthwise convolution over a sequence: forward,
// backward, one-token step.
//
// Bound by memory (bf16: 4 bytes an element forward, 6 backward, against 2 K + 6
// operations and two SFU ones).  A thread takes VEC adjacent channels and a
// segment of the sequence and slides the K-step window over it in registers, so
// each input row is read once but for the K - 1 rows in front of a segment; the
// next rows' loads are issued before the current ones are used.  Measured (B200,
// b = 8, L = 2048, d = 1536, K = 4, us): bf16 forward 23, backward 48 (floors 15 and 23
// at the copy bandwidth), fp32 37 and 62.  What bf16 is bound by: instructions and
// the SFU pipe, which also rounds to bf16 (50 % full forward).  Threads of a CTA:
// `lanes` channel groups (a power of two, at most 32) x 256 / lanes segments.
#pragma once

#include <type_traits>

#include "block_common.cuh"

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
  int lanes;         // channel groups of a CTA
  int ctiles;        // CTAs across the channels; blockIdx.x counts them first
  int T;             // steps of a segment, a multiple of kConvRows
  int64_t segs;      // segments of a sequence
};

struct ConvBwdParams {
  ConvParams f;
  const void *dy;
  int64_t dy_ld;
  void *dx;
  int64_t dx_ld;
  int parts;    // CTAs along the segments
  float *part;  // (parts, d (K + 1)): sums of dweight, then dbias
};

constexpr int kConvThreads = 256;
// Channels a thread takes and rows it loads at a time, forward and backward, and
// the CTAs of 256 threads an SM holds.  Measured (B200, bf16, b = 8, L = 2048, d =
// 1536, K = 4, us): forward 4 x 4 23.2, 2 x 8 24.8, 2 x 4 31.5; with 4 CTAs 26.2,
// 2 30.2.  Backward 2 x 4 48.8 (3 CTAs, 80 registers), 2 x 8 67.7, 4 x 4 93.6 (the
// registers of weight, window, dx and dweight, 4 K a channel, spill); fp32 2 x 4
// 68.2 with 3 CTAs, 63.1 with 2; K = 8 takes 2 either way.
constexpr int kConvVec = 4, kConvRows = 4;
constexpr int kConvBwdVec = 2, kConvBwdRows = 4;
constexpr int conv_fwd_occ(int K) { return K <= 4 ? 3 : 2; }
constexpr int conv_bwd_occ(int K, size_t es) { return K <= 4 && es == 2 ? 3 : 2; }

// The window's entry for step t < 0 of sequence i, channel c.
template <typename T, int K>
__device__ __forceinline__ float win_at(const ConvParams &p, int64_t i, int64_t t, int64_t c) {
  if (!p.win) return 0.0f;
  const int64_t k = (i * p.d + c) * K + K + t, n = p.b * p.d * K;
  return in_bounds(k, n, kBndWork) ? Elem<T>::load(static_cast<const T *>(p.win), k) : 0.0f;
}

__device__ __forceinline__ bool starts_at(const uint8_t *start, int64_t r, int64_t n) {
  return in_bounds(r, n, kBndAct) && start[r] != 0;
}

// Bits of the steps a sequence starts at among `n` (at most N) from row r of the
// `rows` on: one word's load where the bytes are aligned.
template <int N>
__device__ __forceinline__ unsigned start_bits(const uint8_t *start, int64_t r, int n, int64_t rows) {
  const uint8_t *s = start + r;
  if (n <= 0 || !in_bounds(r, rows - ((n < N ? n : N) - 1), kBndAct)) return 0;
  static_assert(N == 4 || N == 8, "one word of start flags");
  using W = typename std::conditional<N == 8, uint2, unsigned>::type;
  unsigned bits = 0;
  if (n >= N && reinterpret_cast<uintptr_t>(s) % N == 0) {
    const W w = *reinterpret_cast<const W *>(s);
    unsigned lo, hi = 0;
    if constexpr (N == 8)
      lo = w.x, hi = w.y;
    else
      lo = w;
    if ((lo | hi) == 0) return 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (lo >> (8 * q) & 0xff) bits |= 1u << q;
      if (N == 8 && (hi >> (8 * q) & 0xff)) bits |= 16u << q;
    }
  } else {
    for (int q = 0; q < N && q < n; ++q)
      if (s[q]) bits |= 1u << q;
  }
  return bits;
}

// Segment k's sequence and position in it.
__device__ __forceinline__ void split_seg(int64_t k, int64_t n, int64_t segs, int64_t &i, int64_t &s) {
  if (n <= 0xffffffffll) {
    const unsigned u = (unsigned)k / (unsigned)segs;
    i = u;
    s = (unsigned)k - u * (unsigned)segs;
  } else {
    i = k / segs;
    s = k - i * segs;
  }
}

// The taps of VEC channels, w[j][e], from their VEC K adjacent values.
template <int K, int VEC>
__device__ __forceinline__ void ld_taps(const ConvParams &p, int64_t c, float (&w)[K][VEC]) {
  alignas(16) float f[VEC * K];
#pragma unroll
  for (int z = 0; z < VEC * K; ++z) f[z] = 0.0f;
  if (in_bounds(c * K, p.d * K - (VEC * K - 1), kBndParam)) {
    const float *s = p.w + c * K;
    if constexpr (VEC > 1 && VEC * K % 4 == 0) {
#pragma unroll
      for (int z = 0; z < VEC * K / 4; ++z)
        reinterpret_cast<float4 *>(f)[z] = __ldg(reinterpret_cast<const float4 *>(s) + z);
    } else {
#pragma unroll
      for (int z = 0; z < VEC * K; ++z) f[z] = __ldg(s + z);
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[j][e] = f[e * K + j];
}

template <typename T, int K, int VEC, bool START>
__global__ void __launch_bounds__(kConvThreads, conv_fwd_occ(K)) conv_fwd_kernel(const ConvParams p) {
  const unsigned tile = blockIdx.x % (unsigned)p.ctiles, blk = blockIdx.x / (unsigned)p.ctiles;
  const int64_t c = (tile * (int64_t)p.lanes + threadIdx.x % p.lanes) * VEC;
  const int64_t k = blk * (int64_t)(kConvThreads / p.lanes) + threadIdx.x / p.lanes;
  if (c >= p.d || k >= p.b * p.segs) return;
  int64_t i, seg;
  split_seg(k, p.b * p.segs, p.segs, i, seg);
  const int64_t t0 = seg * p.T, row = i * p.L;
  const int64_t t1 = t0 + p.T < p.L ? t0 + p.T : p.L;
  const int64_t xn = extent(p.b * p.L, p.d, p.x_ld), yn = extent(p.b * p.L, p.d, p.y_ld);
  using W = typename VecWord<T, VEC>::type;

  float w[K][VEC], bias[VEC];
  ld_taps<K, VEC>(p, c, w);
#pragma unroll
  for (int e = 0; e < VEC; ++e) bias[e] = p.bias ? ld_param(p.bias, c + e, p.d) : 0.0f;
  // v[j]: step t - K + 1 + j in front of each row, v[K - 1 ..] the rows in flight
  float v[K - 1 + kConvRows][VEC];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int64_t t = t0 - K + 1 + j;
    if (START && t >= 0 && starts_at(p.start, row + t, p.b * p.L)) {
#pragma unroll
      for (int q = 0; q < K - 1; ++q)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (q < j) v[q][e] = 0.0f;
    }
    if (t >= 0)
      unpack(ld_raw_ro<T, VEC>(p.x, (row + t) * p.x_ld + c, xn), v[j]);
    else
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = win_at<T, K>(p, i, t, c + e);
  }
  if (t0 == 0 && p.win_out) {  // this thread alone reads this window: it may be in place
    int64_t last = -K;         // the last step a sequence starts at, of those that matter
    if (START)
      for (int64_t t = p.L - 1; t >= 0 && t > p.L - 1 - K && last < 0; --t)
        if (starts_at(p.start, row + t, p.b * p.L)) last = t;
    bool old = true;  // whether the old window reaches past the last step
    if (START)
      for (int64_t t = 0; t < p.L && t < K; ++t) old = old && !starts_at(p.start, row + t, p.b * p.L);
#pragma unroll 1
    for (int e = 0; e < VEC; ++e) {
      float o[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int64_t t = p.L - K + j;
        o[j] = 0.0f;
        if (t >= 0 ? t >= last : old && t >= -K)
          o[j] = t >= 0 ? Elem<T>::load(static_cast<const T *>(p.x), (row + t) * p.x_ld + c + e)
                        : win_at<T, K>(p, i, t, c + e);
      }
      const int64_t q = (i * p.d + c + e) * K;
      if (in_bounds(q, p.b * p.d * K - (K - 1), kBndWork)) {
#pragma unroll
        for (int j = 0; j < K; ++j) Elem<T>::store(static_cast<T *>(p.win_out), q + j, o[j]);
      }
    }
  }

  const T *xp = static_cast<const T *>(p.x) + (row + t0) * p.x_ld + c;
  int64_t sr = row + t0;  // row of the next start flags
  W raw[kConvRows];
  unsigned st = 0;  // bit q: a sequence starts at row q
  const auto load = [&](int n) {  // the next rows, of which n are the segment's
#pragma unroll
    for (int q = 0; q < kConvRows; ++q) {
      raw[q] = W{};
      if (q < n) raw[q] = ld_raw_ro<T, VEC>(p.x, xp + q * p.x_ld - static_cast<const T *>(p.x), xn);
    }
    xp += kConvRows * p.x_ld;
    if (START) {
      st = start_bits<kConvRows>(p.start, sr, n, p.b * p.L);
      sr += kConvRows;
    }
  };
  int64_t yo = (row + t0) * p.y_ld + c;
  int left = (int)(t1 - t0);
  W cur[kConvRows];
  unsigned cst = 0;
  // PLAIN: whole rows of the segment, no sequence starting
  const auto rows = [&](auto plain) {
    constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
    for (int q = 0; q < kConvRows; ++q) {
      unpack(cur[q], v[K - 1 + q]);
      if (START && !PLAIN && (cst >> q & 1)) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[q + j][e] = 0.0f;
      }
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = bias[e];
#pragma unroll
      for (int j = 0; j < K; ++j) fma_vec<VEC>(o, w[j], v[q + j]);
      if (p.silu) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = silu_f32(o[e]);
      }
      if (PLAIN || q < left) st_vec<T, VEC>(p.y, yo + q * p.y_ld, yn, o);
    }
  };
  load(left);
  for (; left > 0; left -= kConvRows) {
#pragma unroll
    for (int q = 0; q < kConvRows; ++q) cur[q] = raw[q];
    cst = st;
    load(left - kConvRows);
    if (left >= kConvRows && cst == 0)
      rows(std::true_type());
    else
      rows(std::false_type());
    yo += kConvRows * p.y_ld;
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = v[kConvRows + j][e];
  }
}

// dx_t = sum_m w[K-1-m] dp_{t+m}, dp = dy act'(p): a segment's thread walks its
// steps and the K - 1 behind them, forming p again from the window.  dweight and
// dbias are summed in registers over the segments a thread takes, then over the
// CTA's segments in shared memory, one partial row per CTA.
template <typename T, int K, int VEC, bool START>
__global__ void __launch_bounds__(kConvThreads, conv_bwd_occ(K, sizeof(T))) conv_bwd_kernel(const ConvBwdParams q) {
  const ConvParams &p = q.f;
  __shared__ float red[kConvThreads * VEC];
  const int lane = threadIdx.x % p.lanes, slot = threadIdx.x / p.lanes;
  const int slots = kConvThreads / p.lanes;
  const unsigned tile = blockIdx.x % (unsigned)p.ctiles, blk = blockIdx.x / (unsigned)p.ctiles;
  const int64_t c = (tile * (int64_t)p.lanes + lane) * VEC;
  const bool on = c < p.d;
  const int64_t R = p.b * p.L;
  const int64_t xn = extent(R, p.d, p.x_ld), gn = extent(R, p.d, q.dy_ld),
                on_ = extent(R, p.d, q.dx_ld);
  using W = typename VecWord<T, VEC>::type;
  constexpr int N = kConvBwdRows;

  float w[K][VEC], bias[VEC], dw[K][VEC], db[VEC];
  ld_taps<K, VEC>(p, on ? c : 0, w);
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = 0.0f;
    bias[e] = on && p.bias ? ld_param(p.bias, c + e, p.d) : 0.0f;
    db[e] = 0.0f;
  }

  for (int64_t k = blk * (int64_t)slots + slot; on && k < p.b * p.segs;
       k += q.parts * (int64_t)slots) {
    int64_t i, seg;
    split_seg(k, p.b * p.segs, p.segs, i, seg);
    const int64_t t0 = seg * p.T, row = i * p.L;
    const int64_t t1 = t0 + p.T < p.L ? t0 + p.T : p.L;          // dx of [t0, t1)
    const int64_t t2 = t1 + K - 1 < p.L ? t1 + K - 1 : p.L;      // dp up to here
    float v[K - 1 + N][VEC], g[K][VEC];  // g[m]: dx of step t - m so far
    int age = 2 * K;                     // steps since the sequence's start, as far as it matters
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int64_t t = t0 - K + 1 + j;
      if (START) {
        const bool st = t >= 0 && starts_at(p.start, row + t, R);
        age = st ? 0 : age + 1;
        if (st) {
#pragma unroll
          for (int z = 0; z < K - 1; ++z)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              if (z < j) v[z][e] = 0.0f;
        }
      }
      if (t >= 0)
        unpack(ld_raw_ro<T, VEC>(p.x, (row + t) * p.x_ld + c, xn), v[j]);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = win_at<T, K>(p, i, t, c + e);
    }
#pragma unroll
    for (int m = 0; m < K; ++m)
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[m][e] = 0.0f;

    // steps [t0, t1 + K - 1); those past the sequence's end have dp = 0 and only
    // let out the last dx
    const T *xp = static_cast<const T *>(p.x) + (row + t0) * p.x_ld + c;
    const T *gp = static_cast<const T *>(q.dy) + (row + t0) * q.dy_ld + c;
    int64_t sr = row + t0;  // row of the next start flags
    const int all = (int)(t2 - t0), mine = (int)(t1 - t0);
    W rx[N], rg[N];
    unsigned st = 0;
    const auto load = [&](int n) {
#pragma unroll
      for (int z = 0; z < N; ++z) {
        rx[z] = rg[z] = W{};
        if (z < n) {
          rx[z] = ld_raw_ro<T, VEC>(p.x, xp + z * p.x_ld - static_cast<const T *>(p.x), xn);
          rg[z] = ld_raw_ro<T, VEC>(q.dy, gp + z * q.dy_ld - static_cast<const T *>(q.dy), gn);
        }
      }
      xp += N * p.x_ld;
      gp += N * q.dy_ld;
      if (START) {
        st = start_bits<N>(p.start, sr, n, R);
        sr += N;
      }
    };
    int64_t o = (row + t0 - (K - 1)) * q.dx_ld + c;
    int t = 0;
    W cx[N], cg[N];
    unsigned cst = 0;
    // PLAIN: all of the rows are the segment's, their dx too, and every tap is
    // its sequence's
    const auto rows = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
      for (int z = 0; z < N; ++z) {
        unpack(cx[z], v[K - 1 + z]);
        if (START && !PLAIN) {
          const bool s = cst >> z & 1;
          age = s ? 0 : age + 1;
          if (s) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
              for (int e = 0; e < VEC; ++e) v[z + j][e] = 0.0f;
          }
        }
        float dp[VEC];
        unpack(cg[z], dp);
        if (p.silu) {
          float s[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[e] = bias[e];
#pragma unroll
          for (int j = 0; j < K; ++j) fma_vec<VEC>(s, w[j], v[z + j]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float sg = sigmoid_f32(s[e]);
            dp[e] *= fmaf(s[e] * sg, 1.0f - sg, sg);
          }
        }
        if (!PLAIN && t + z >= all) {  // past the end: p may be anything
#pragma unroll
          for (int e = 0; e < VEC; ++e) dp[e] = 0.0f;
        }
#pragma unroll
        for (int m = K - 1; m > 0; --m)
#pragma unroll
          for (int e = 0; e < VEC; ++e) g[m][e] = g[m - 1][e];
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[0][e] = 0.0f;
#pragma unroll
        for (int m = 0; m < K; ++m)
          if (PLAIN || !START || m <= age) fma_vec<VEC>(g[m], w[K - 1 - m], dp);
        if (PLAIN || t + z < mine) {
#pragma unroll
          for (int m = 0; m < K; ++m)
            if (PLAIN || !START || m <= age) fma_vec<VEC>(dw[K - 1 - m], v[z + K - 1 - m], dp);
#pragma unroll
          for (int e = 0; e < VEC; ++e) db[e] += dp[e];
        }
        if (PLAIN || (t + z >= K - 1 && t + z < mine + K - 1))
          st_vec<T, VEC>(q.dx, o + z * q.dx_ld, on_, g[K - 1]);
      }
      if (START && PLAIN) age += N;
    };
    load(all);
    for (; t < mine + K - 1; t += N) {
#pragma unroll
      for (int z = 0; z < N; ++z) cx[z] = rx[z], cg[z] = rg[z];
      cst = st;
      load(all - t - N);
      if (t >= K - 1 && t + N <= mine && cst == 0 && (!START || age >= K - 2))
        rows(std::true_type());
      else
        rows(std::false_type());
      o += N * q.dx_ld;
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[j][e] = v[N + j][e];
    }
  }

  // over the CTA's segments, in order
  float *part = q.part + blk * (p.d * (K + 1));
  const int64_t pn = p.d * (K + 1);
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) red[threadIdx.x * VEC + e] = j < K ? dw[j][e] : db[e];
    __syncthreads();
    // thread (lane, e) of the first lanes * VEC sums its column over the slots
    for (int z = threadIdx.x; z < p.lanes * VEC; z += kConvThreads) {
      const int64_t cc = tile * (int64_t)p.lanes * VEC + z;
      if (cc >= p.d) continue;
      float s = 0.0f;
      for (int r = 0; r < slots; ++r) s += red[r * p.lanes * VEC + z];
      const int64_t o = j < K ? cc * K + j : p.d * K + cc;
      if (in_bounds(o, pn, kBndWork)) part[o] = s;
    }
  }
}

// N elements (adjacent in memory and in a register array) as 16-byte accesses
// where their bytes are whole ones of those.
template <typename T, int N> __device__ __forceinline__ void ld_span(const T *p, T *v) {
  constexpr int B = N * (int)sizeof(T);
  if constexpr (B % 16 == 0) {
#pragma unroll
    for (int z = 0; z < B / 16; ++z)
      reinterpret_cast<uint4 *>(v)[z] = reinterpret_cast<const uint4 *>(p)[z];
  } else {
#pragma unroll
    for (int z = 0; z < N; ++z) v[z] = p[z];
  }
}
template <typename T, int N> __device__ __forceinline__ void st_span(T *p, const T *v) {
  constexpr int B = N * (int)sizeof(T);
  if constexpr (B % 16 == 0) {
#pragma unroll
    for (int z = 0; z < B / 16; ++z)
      reinterpret_cast<uint4 *>(p)[z] = reinterpret_cast<const uint4 *>(v)[z];
  } else {
#pragma unroll
    for (int z = 0; z < N; ++z) p[z] = v[z];
  }
}

// One token: VEC channels a thread, whose windows and taps are VEC K adjacent
// elements each.  VEC > 1 needs 16-byte aligned windows, weights and rows.
template <typename T, int K, int VEC>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvParams p, void *win) {
  const int64_t G = p.d / VEC;
  const int64_t k = blockIdx.x * (int64_t)kConvThreads + threadIdx.x;
  if (k >= p.b * G) return;
  const int64_t i = p.b * G <= 0x7fffffff ? (int64_t)((unsigned)k / (unsigned)G) : k / G;
  const int64_t c = (k - i * G) * VEC, q = (i * p.d + c) * K;
  alignas(16) T v[VEC * K];
  alignas(16) float w[VEC * K];
  float x[VEC], o[VEC];
  T *wp = static_cast<T *>(win) + q;
  const bool ok = in_bounds(q, p.b * p.d * K - (VEC * K - 1), kBndWork) &&
                  in_bounds(c * K, p.d * K - (VEC * K - 1), kBndParam);
  if (!ok) return;
  ld_span<T, VEC * K>(wp, v);
  ld_span<float, VEC * K>(p.w + c * K, w);
  unpack(ld_raw_ro<T, VEC>(p.x, i * p.x_ld + c, extent(p.b, p.d, p.x_ld)), x);
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = p.bias ? ld_param(p.bias, c + e, p.d) : 0.0f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) v[e * K + j] = v[e * K + j + 1];
    if constexpr (sizeof(T) == 2)
      v[e * K + K - 1] = __float2bfloat16_rn(x[e]);  // exact: x came from bf16
    else
      v[e * K + K - 1] = x[e];
#pragma unroll
    for (int j = 0; j < K; ++j) o[e] = fmaf(w[e * K + j], static_cast<float>(v[e * K + j]), o[e]);
    if (p.silu) o[e] = silu_f32(o[e]);
  }
  st_span<T, VEC * K>(wp, v);
  st_vec<T, VEC>(p.y, i * p.y_ld + c, extent(p.b, p.d, p.y_ld), o);
}

}  // namespace ssm
