// block_ops.cu -- the C ABI of the operators around the scan (gated
// recurrence, causal convolution, norms): argument validation, kernel
// selection and launch, under the rules of ssmscan.cu.
#include <cmath>
#include <type_traits>
#include <utility>

#include "abi_host.cuh"
#include "conv1d.cuh"
#include "gated_scan.cuh"
#include "norms.cuh"

using namespace ssm_host;

namespace {

cudaStream_t cu(ssm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// A named argument as rows of `width` bytes, `pitch` bytes apart; contiguous
// arguments are one row.
struct RowSpan {
  const char *name;
  const void *p;
  int64_t rows, width, pitch;
};

// Whether two arguments share a byte.  Rows of the same pitch may interleave
// (the two halves of one projection's rows).
bool rows_overlap(const RowSpan &a, const RowSpan &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (uintptr_t)((a.rows - 1) * a.pitch + a.width);
  const uintptr_t b1 = b0 + (uintptr_t)((b.rows - 1) * b.pitch + b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t off = a0 <= b0 ? (int64_t)((b0 - a0) % (uintptr_t)a.pitch)
                               : (a.pitch - (int64_t)((a0 - b0) % (uintptr_t)a.pitch)) % a.pitch;
  return off < a.width || a.pitch - off < b.width;
}

// Collects a call's arguments and checks them: presence, alignment, strides,
// and that no output shares bytes with another argument.
class Args {
 public:
  Args(const char *what, size_t es) : what_(what), es_(es) {}
  // `rows` rows of `d` elements of `es` bytes, ld elements apart
  void rows(bool out, const char *name, const void *p, int64_t rows, int64_t d, int64_t ld,
            size_t es = 0) {
    es = es ? es : es_;
    if (!p) return;
    if (status_ == SSM_OK && !aligned(p, es))
      status_ = fail(SSM_ERR_INVALID_ARG, "%s: %s is not %zu-byte aligned", what_, name, es);
    int64_t t;
    if (status_ == SSM_OK && ld >= (int64_t)1 << 31)
      status_ = fail(SSM_ERR_INVALID_ARG, "%s: %s_ld %lld is not below 2^31", what_, name, (long long)ld);
    if (status_ == SSM_OK && ld < d)
      status_ = fail(SSM_ERR_INVALID_ARG, "%s: %s_ld %lld is below the row's %lld elements", what_,
                     name, (long long)ld, (long long)d);
    if (status_ == SSM_OK && (!mul_ok(rows, ld, &t) || t > INT64_MAX / 16))
      status_ = fail(SSM_ERR_INVALID_ARG, "%s: the rows of %s overflow int64", what_, name);
    add(out, {name, p, rows, d * (int64_t)es, ld * (int64_t)es});
  }
  void flat(bool out, const char *name, const void *p, int64_t bytes, size_t align = 4) {
    if (!p) return;
    if (status_ == SSM_OK && !aligned(p, align))
      status_ = fail(SSM_ERR_INVALID_ARG, "%s: %s is not %zu-byte aligned", what_, name, align);
    add(out, {name, p, 1, bytes, bytes});
  }
  // this output may be exactly this input
  void same(const char *out, const char *in) {
    same_out_ = out;
    same_in_ = in;
  }
  ssm_status check() {
    if (status_ != SSM_OK) return status_;
    for (int i = 0; i < n_; ++i) {
      if (!out_[i]) continue;
      for (int j = 0; j < n_; ++j) {
        if (j == i || (out_[j] && j < i)) continue;
        const RowSpan &a = span_[i], &b = span_[j];
        if (same_out_ && !strcmp(a.name, same_out_) && !strcmp(b.name, same_in_) && a.p == b.p &&
            a.rows == b.rows && a.width == b.width && a.pitch == b.pitch)
          continue;
        if (rows_overlap(a, b))
          return fail(SSM_ERR_INVALID_ARG, "%s: %s overlaps %s", what_, a.name, b.name);
      }
    }
    return SSM_OK;
  }

 private:
  void add(bool out, const RowSpan &s) {
    if (n_ == kMax) {
      status_ = fail(SSM_ERR_INVALID_ARG, "%s: too many arguments", what_);
      return;
    }
    out_[n_] = out;
    span_[n_++] = s;
  }
  static constexpr int kMax = 32;
  const char *what_;
  size_t es_;
  ssm_status status_ = SSM_OK;
  int n_ = 0;
  bool out_[kMax];
  RowSpan span_[kMax];
  const char *same_out_ = nullptr, *same_in_ = nullptr;
};

ssm_status bad_dtype(const char *what, ssm_dtype t) {
  return t == SSM_F32 || t == SSM_BF16 ? SSM_OK
                                       : fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", what, (int)t);
}

// Sizes of a call: none negative, their product (times 16 bytes) in int64.
bool sizes_ok(std::initializer_list<int64_t> sizes) {
  int64_t t = 16;
  for (int64_t s : sizes) {
    if (s < 0) return false;
    if (s > 0 && !mul_ok(t, s, &t)) return false;
  }
  return true;
}

ssm_status zero(float *p, int64_t n, cudaStream_t st, const char *what) {
  if (!p || n <= 0) return SSM_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)n * 4, st);
  return e == cudaSuccess ? SSM_OK : fail(SSM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

ssm_status need_workspace(const char *what, const void *ws, size_t have, size_t need) {
  if (need == 0) return SSM_OK;
  if (!ws || have < need)
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, ws ? have : 0, need);
  return SSM_OK;
}

// The parameters' gradients from n partial rows of m0 + m1 + m2 values.
ssm_status col_sum(const float *part, int64_t n, int64_t m0, float *out0, int64_t m1, float *out1,
                   int64_t m2, float *out2, cudaStream_t st, const char *what) {
  const dim3 block(ssm::kColSumCols, ssm::kColSumRows);
  const int64_t m = m0 + m1 + m2;
  // may start while the kernel that writes the partial rows ends
  return launch_dependent(ssm::col_sum_kernel, dim3((unsigned)((m + ssm::kColSumCols - 1) / ssm::kColSumCols)),
                          block, 0, st, what, ssm::ColSumParams{part, n, m0, m1, m2, out0, out1, out2});
}

__global__ void copy_or_zero_f32(const float *src, float *dst, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    dst[i] = src ? src[i] : 0.0f;
}

// An empty sequence hands its start state (or zeros) through.
ssm_status pass_state(const float *src, float *dst, int64_t n, cudaStream_t st, const char *what) {
  if (!dst || src == dst || n <= 0) return SSM_OK;
  copy_or_zero_f32<<<grid_for(n), 256, 0, st>>>(src, dst, n);
  return check_launch(what);
}

// A row stride as the gated kernels take it; -1, which the argument check
// refuses (as below the row), where it is not below 2^31.
int ld32(int64_t ld) { return ld >= 0 && ld <= 0x7fffffff ? (int)ld : -1; }

constexpr int64_t kMaxGrid = 0x7fffffff;

// Whether rows of T can be read VEC elements at a time.
bool vec_rows(int64_t vec, size_t es, int64_t d, std::initializer_list<std::pair<const void *, int64_t>> rows) {
  if (d % vec != 0) return false;
  for (const auto &r : rows)
    if (r.first && (!aligned(r.first, vec * es) || r.second % vec != 0)) return false;
  return true;
}

// --------------------------------------------------------- gated recurrence
int64_t gated_chunks(int64_t L) { return (L + ssm::kGatedChunk - 1) / ssm::kGatedChunk; }

// Parts of a warp (S) and CTAs of a cluster (C).  A CTA's round is 64 S steps of
// 1 / S of the channels, the same work whatever S (the bf16 backward's is 32 S steps).
// The rule is the forward's, and the backward, which holds 2 CTAs an SM of either
// type, takes the same plan.  In tenths of a microsecond, as measured: a round takes 14 with one CTA on an
// SM, 24 with as many as it holds (2 of bf16, 3 of fp32); clusters, whose CTAs wait
// for each other in every round, take a third more; a CTA of 32 bytes of a row (S =
// 4) a fifth more than one of 64, one of 128 a tenth less.  bf16, b = 8, L = 2048, d
// = 1536, when this was fitted (us): S = 2 61, S = 1 70, S = 4 70, S = 1 in clusters
// of 2 81; b = 1, L = 16384, d = 64: S = 2 178, S = 4 107, S = 4 in clusters of 8 24.
struct GatedPlan {
  int parts, ctiles, csize;
};
GatedPlan gated_plan(int64_t b, int64_t L, int64_t d, size_t es) {
  const int64_t sms = device_sms(), holds = es == 2 ? 2 : 3;
  GatedPlan best{1, 1, 1};
  int64_t least = -1;
  for (int s = 1; s <= 4; s *= 2)
    for (int c = 1; c <= ssm::kGatedMaxCluster; c *= 2) {
      const int64_t channels = 128 / (int64_t)es / s;
      const int64_t tiles = (d + channels - 1) / channels, ctas = b * tiles * c;
      const int64_t rounds = (L + 64 * s * c - 1) / (64 * s * c);
      const int64_t waves = ctas / (holds * sms), rest = ctas % (holds * sms);
      const int64_t wave = waves * 24 + (rest == 0 ? 0 : 14 + 10 * ((rest + sms - 1) / sms - 1) / (holds - 1));
      const int64_t cost = rounds * wave * (c > 1 ? 4 : 3) * (s == 1 ? 9 : s == 2 ? 10 : 12);
      if (least < 0 || cost < least) {
        least = cost;
        best = GatedPlan{s, (int)tiles, c};
      }
    }
  return best;
}
int64_t gated_bwd_parts(int64_t b, int64_t L, int64_t d) {  // of whichever type
  const int f = gated_plan(b, L, d, 4).csize, h = gated_plan(b, L, d, 2).csize;
  return b * (f > h ? f : h);
}

template <auto Kernel, typename P>
ssm_status launch_gated(const P &p, int64_t b, const GatedPlan &g, int smem, int most, cudaStream_t st,
                        const char *what) {
  // the most any call of this kernel takes, set once
  if (ssm_status s = ensure_smem<Kernel>(most, what)) return s;
  if (b > kMaxGrid / ((int64_t)g.ctiles * g.csize))
    return fail(SSM_ERR_UNSUPPORTED, "%s: b * d_in too large for one grid", what);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(b * g.ctiles * g.csize));
  cfg.blockDim = dim3(ssm::kGatedThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)g.csize;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, Kernel, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(SSM_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
  }
  return ok();
}

template <typename T, bool ASYNC, bool GATE>
ssm_status gated_fwd_t(ssm::GatedParams p, cudaStream_t st) {
  const GatedPlan g = gated_plan(p.b, p.L, p.d, sizeof(T));
  p.parts = g.parts, p.ctiles = g.ctiles, p.csize = g.csize;
  const int smem = ssm::gated_smem(GATE ? 4 : 3, ssm::kGatedFwdSteps, g.csize);
  constexpr int most = ssm::gated_smem(GATE ? 4 : 3, ssm::kGatedFwdSteps, ssm::kGatedMaxCluster);
  if (p.start)
    return launch_gated<ssm::gated_fwd_kernel<T, ASYNC, GATE, true>>(p, p.b, g, smem, most, st, "ssm_gated_scan_fwd");
  return launch_gated<ssm::gated_fwd_kernel<T, ASYNC, GATE, false>>(p, p.b, g, smem, most, st, "ssm_gated_scan_fwd");
}
template <typename T, bool ASYNC, bool GATE>
ssm_status gated_bwd_t(ssm::GatedBwdParams q, int64_t *parts, cudaStream_t st) {
  const GatedPlan g = gated_plan(q.f.b, q.f.L, q.f.d, sizeof(T));
  q.f.parts = g.parts, q.f.ctiles = g.ctiles, q.f.csize = g.csize;
  *parts = q.f.b * g.csize;
  const int smem = ssm::gated_smem(GATE ? 5 : 4, ssm::gated_bwd_steps<T>(), g.csize);
  constexpr int most = ssm::gated_smem(GATE ? 5 : 4, ssm::gated_bwd_steps<T>(), ssm::kGatedMaxCluster);
  if (q.f.start)
    return launch_gated<ssm::gated_bwd_kernel<T, ASYNC, GATE, true>>(q, q.f.b, g, smem, most, st, "ssm_gated_scan_bwd");
  return launch_gated<ssm::gated_bwd_kernel<T, ASYNC, GATE, false>>(q, q.f.b, g, smem, most, st, "ssm_gated_scan_bwd");
}
// Rows in 16-byte pieces (inputs) and VEC elements (outputs) where all allow it.
template <typename T> ssm_status gated_fwd_any(const ssm::GatedParams &p, cudaStream_t st) {
  const bool v = vec_rows(16 / sizeof(T), sizeof(T), p.d,
                          {{p.u, p.u_ld}, {p.ga, p.ga_ld}, {p.gx, p.gx_ld}, {p.z, p.z_ld}}) &&
                 vec_rows(ssm::gated_vec<T>(), sizeof(T), p.d, {{p.y, p.y_ld}});
  if (p.z) return v ? gated_fwd_t<T, true, true>(p, st) : gated_fwd_t<T, false, true>(p, st);
  return v ? gated_fwd_t<T, true, false>(p, st) : gated_fwd_t<T, false, false>(p, st);
}
template <typename T>
ssm_status gated_bwd_any(const ssm::GatedBwdParams &q, int64_t *parts, cudaStream_t st) {
  const ssm::GatedParams &p = q.f;
  const bool v = vec_rows(16 / sizeof(T), sizeof(T), p.d,
                          {{p.u, p.u_ld}, {p.ga, p.ga_ld}, {p.gx, p.gx_ld}, {p.z, p.z_ld},
                           {q.dout, q.dout_ld}}) &&
                 vec_rows(ssm::gated_vec<T>(), sizeof(T), p.d,
                          {{q.du, q.du_ld}, {q.dga, q.dga_ld}, {q.dgx, q.dgx_ld}, {q.dz, q.dz_ld}});
  if (p.z) return v ? gated_bwd_t<T, true, true>(q, parts, st) : gated_bwd_t<T, false, true>(q, parts, st);
  return v ? gated_bwd_t<T, true, false>(q, parts, st) : gated_bwd_t<T, false, false>(q, parts, st);
}
template <typename T, int VEC>
ssm_status gated_step_v(const ssm::GatedParams &p, float *state, cudaStream_t st) {
  const int64_t blocks = (p.b * (p.d / VEC) + 255) / 256;
  if (blocks > kMaxGrid)
    return fail(SSM_ERR_UNSUPPORTED, "ssm_gated_state_update: b * d_in too large for one grid");
  if (p.z)
    ssm::gated_step_kernel<T, VEC, true><<<(unsigned)blocks, 256, 0, st>>>(p, state);
  else
    ssm::gated_step_kernel<T, VEC, false><<<(unsigned)blocks, 256, 0, st>>>(p, state);
  return check_launch("ssm_gated_state_update");
}
template <typename T>
ssm_status gated_step_any(const ssm::GatedParams &p, float *state, cudaStream_t st) {
  if (vec_rows(4, sizeof(T), p.d, {{p.u, p.u_ld}, {p.ga, p.ga_ld}, {p.gx, p.gx_ld}, {p.z, p.z_ld},
                                   {p.y, p.y_ld}}) && aligned(state, 16))
    return gated_step_v<T, 4>(p, state, st);
  return gated_step_v<T, 1>(p, state, st);
}

ssm_status check_gated(const char *what, Args &a, const ssm::GatedParams &p, ssm_dtype dtype) {
  if (ssm_status s = bad_dtype(what, dtype)) return s;
  if (!sizes_ok({p.b, p.L, p.d}))
    return fail(SSM_ERR_INVALID_ARG, "%s: negative size or sizes that overflow int64", what);
  if (p.L > (1 << 30)) return fail(SSM_ERR_UNSUPPORTED, "%s: L above 2^30", what);
  const int64_t R = p.b * p.L;
  if (R > 0 && p.d > 0 && (!p.u || !p.ga || !p.gx || !p.A))
    return fail(SSM_ERR_INVALID_ARG, "%s: u, gate_a, gate_x and A are required", what);
  a.rows(false, "u", p.u, R, p.d, p.u_ld);
  a.rows(false, "gate_a", p.ga, R, p.d, p.ga_ld);
  a.rows(false, "gate_x", p.gx, R, p.d, p.gx_ld);
  a.rows(false, "z", p.z, R, p.d, p.z_ld);
  a.flat(false, "A", p.A, p.d * 4);
  a.flat(false, "bias_a", p.ba, p.d * 4);
  a.flat(false, "bias_x", p.bx, p.d * 4);
  a.flat(false, "seq_start", p.start, R, 1);
  return SSM_OK;
}

ssm_status check_states(const char *what, const void *p, size_t have, int64_t b, int64_t L, int64_t d) {
  const size_t need = (size_t)(b * gated_chunks(L) * d) * 4;
  if (have < need)
    return fail(SSM_ERR_WORKSPACE, "%s: chunk_states of %zu bytes, %zu needed", what, have, need);
  (void)p;
  return SSM_OK;
}

// -------------------------------------------------------------- convolution
// Shape of the convolution's CTAs: `lanes` channel groups of VEC that fit a
// warp, 256 / lanes segments of T steps.  A CTA's time goes as T plus the rows a
// segment reads of its neighbours and its prologue (some 16 rows' worth), so T is
// the multiple of 8 with the least of it over the waves of `occ` CTAs an SM.
// Backward the CTAs of one wave loop over the segments instead, since each
// writes a partial row of the parameters' gradients.
struct ConvPlan {
  int lanes, T;
  int64_t ctiles, segs, blocks;  // blocks: CTAs along the segments
};
ConvPlan conv_plan(int64_t b, int64_t L, int64_t d, int vec, int occ, bool one_wave) {
  ConvPlan best{};
  int64_t least = -1;
  ConvPlan c{};
  const int64_t G = d > 0 ? (d + vec - 1) / vec : 1;
  c.lanes = 1;
  while (c.lanes < 32 && c.lanes < G) c.lanes *= 2;
  c.ctiles = (G + c.lanes - 1) / c.lanes;
  const int64_t slots = ssm::kConvThreads / c.lanes;
  const int64_t room = occ * (int64_t)device_sms();
  const int64_t parts = room / c.ctiles > 0 ? room / c.ctiles : 1;
  for (c.T = 8; c.T <= 128; c.T += 8) {
    c.segs = L > 0 ? (L + c.T - 1) / c.T : 1;
    c.blocks = (b * c.segs + slots - 1) / slots;
    int64_t waves;
    if (one_wave) {
      waves = c.blocks > 0 ? (c.blocks + parts - 1) / parts : 1;
      c.blocks = (c.blocks + waves - 1) / waves;
      if (parts == 1) waves *= (c.ctiles + room - 1) / room;
    } else {
      waves = (c.blocks * c.ctiles + room - 1) / room;
    }
    const int64_t cost = waves * (c.T + 16);
    if (least < 0 || cost < least) least = cost, best = c;
  }
  return best;
}
int64_t conv_bwd_parts(int64_t b, int64_t L, int64_t d) {  // of whichever kernel the call takes
  int64_t most = 0;
  for (int vec : {1, ssm::kConvBwdVec})
    for (int occ : {2, 3}) {
      const int64_t n = conv_plan(b, L, d, vec, occ, true).blocks;
      if (n > most) most = n;
    }
  return most;
}

template <typename T, int K, int VEC>
ssm_status launch_conv_fwd(ssm::ConvParams p, cudaStream_t st) {
  const ConvPlan c = conv_plan(p.b, p.L, p.d, VEC, ssm::conv_fwd_occ(K), false);
  if (c.blocks > kMaxGrid / c.ctiles)
    return fail(SSM_ERR_UNSUPPORTED, "ssm_conv1d_fwd: b * L * d_in too large for one grid");
  p.lanes = c.lanes, p.ctiles = (int)c.ctiles, p.T = c.T, p.segs = c.segs;
  const unsigned grid = (unsigned)(c.blocks * c.ctiles);
  if (p.start)
    ssm::conv_fwd_kernel<T, K, VEC, true><<<grid, ssm::kConvThreads, 0, st>>>(p);
  else
    ssm::conv_fwd_kernel<T, K, VEC, false><<<grid, ssm::kConvThreads, 0, st>>>(p);
  return check_launch("ssm_conv1d_fwd");
}

template <typename T, int K, int VEC>
ssm_status launch_conv_bwd(ssm::ConvBwdParams q, int64_t *parts, cudaStream_t st) {
  const ConvPlan c = conv_plan(q.f.b, q.f.L, q.f.d, VEC, ssm::conv_bwd_occ(K, sizeof(T)), true);
  if (c.blocks > kMaxGrid / c.ctiles)
    return fail(SSM_ERR_UNSUPPORTED, "ssm_conv1d_bwd: b * L * d_in too large for one grid");
  q.f.lanes = c.lanes, q.f.ctiles = (int)c.ctiles, q.f.T = c.T, q.f.segs = c.segs;
  q.parts = (int)c.blocks;
  *parts = c.blocks;
  const unsigned grid = (unsigned)(c.blocks * c.ctiles);
  if (q.f.start)
    ssm::conv_bwd_kernel<T, K, VEC, true><<<grid, ssm::kConvThreads, 0, st>>>(q);
  else
    ssm::conv_bwd_kernel<T, K, VEC, false><<<grid, ssm::kConvThreads, 0, st>>>(q);
  return check_launch("ssm_conv1d_bwd");
}

template <typename T, int K, int VEC>
ssm_status launch_conv_step(const ssm::ConvParams &p, void *win, cudaStream_t st) {
  const int64_t n = p.b * (p.d / VEC), blocks = (n + ssm::kConvThreads - 1) / ssm::kConvThreads;
  if (blocks > kMaxGrid)
    return fail(SSM_ERR_UNSUPPORTED, "ssm_conv1d_update: b * d_in too large for one grid");
  ssm::conv_step_kernel<T, K, VEC><<<(unsigned)blocks, ssm::kConvThreads, 0, st>>>(p, win);
  return check_launch("ssm_conv1d_update");
}

template <typename T, int K>
ssm_status conv_fwd_k(const ssm::ConvParams &p, cudaStream_t st) {
  constexpr int VEC = ssm::kConvVec;
  if (vec_rows(VEC, sizeof(T), p.d, {{p.x, p.x_ld}, {p.y, p.y_ld}}) && aligned(p.w, 16))
    return launch_conv_fwd<T, K, VEC>(p, st);
  return launch_conv_fwd<T, K, 1>(p, st);
}
template <typename T, int K>
ssm_status conv_bwd_k(const ssm::ConvBwdParams &q, int64_t *parts, cudaStream_t st) {
  constexpr int VEC = ssm::kConvBwdVec;
  if (vec_rows(VEC, sizeof(T), q.f.d, {{q.f.x, q.f.x_ld}, {q.dy, q.dy_ld}, {q.dx, q.dx_ld}}) &&
      aligned(q.f.w, 16))
    return launch_conv_bwd<T, K, VEC>(q, parts, st);
  return launch_conv_bwd<T, K, 1>(q, parts, st);
}
template <typename T, int K>
ssm_status conv_step_k(const ssm::ConvParams &p, void *win, cudaStream_t st) {
  if (vec_rows(4, sizeof(T), p.d, {{p.x, p.x_ld}, {p.y, p.y_ld}}) && aligned(win, 16) && aligned(p.w, 16))
    return launch_conv_step<T, K, 4>(p, win, st);
  return launch_conv_step<T, K, 1>(p, win, st);
}

// f.template operator()<T, K>() for the call's type and width
template <typename F> ssm_status conv_dispatch(ssm_dtype t, int64_t K, F &&f) {
  const auto by_k = [&](auto type) -> ssm_status {
    switch (K) {
      case 1: return f(type, std::integral_constant<int, 1>());
      case 2: return f(type, std::integral_constant<int, 2>());
      case 3: return f(type, std::integral_constant<int, 3>());
      case 4: return f(type, std::integral_constant<int, 4>());
      case 5: return f(type, std::integral_constant<int, 5>());
      case 6: return f(type, std::integral_constant<int, 6>());
      case 7: return f(type, std::integral_constant<int, 7>());
      default: return f(type, std::integral_constant<int, 8>());
    }
  };
  return t == SSM_BF16 ? by_k(__nv_bfloat16()) : by_k(float());
}

ssm_status check_conv(const char *what, Args &a, const ssm::ConvParams &p, int64_t K,
                      ssm_dtype dtype) {
  if (ssm_status s = bad_dtype(what, dtype)) return s;
  if (K < 1 || K > ssm::kMaxConv)
    return fail(SSM_ERR_UNSUPPORTED, "%s: d_conv %lld not in 1 .. %d", what, (long long)K, ssm::kMaxConv);
  if (!sizes_ok({p.b, p.L, p.d, K}))
    return fail(SSM_ERR_INVALID_ARG, "%s: negative size or sizes that overflow int64", what);
  const int64_t R = p.b * p.L;
  if (R > 0 && p.d > 0 && (!p.x || !p.w))
    return fail(SSM_ERR_INVALID_ARG, "%s: x and weight are required", what);
  a.rows(false, "x", p.x, R, p.d, p.x_ld);
  a.flat(false, "weight", p.w, p.d * K * 4);
  a.flat(false, "bias", p.bias, p.d * 4);
  a.flat(false, "seq_start", p.start, R, 1);
  return SSM_OK;
}

// -------------------------------------------------------------------- norms
// Threads of a row of nv vectors and vectors of a thread (1 .. 4): the pair with
// the fewest idle places, of those the one with the most vectors a thread, whose
// loads are in flight together (bf16, 16384 x 1536, forward: 3 a thread 33 us, 2
// 35, 1 47; backward 60, 70, 105).  Where all rows together do not fill the device,
// the fewest vectors a thread instead (64 rows: 2.5 us against 3.2).  tpr = 0: longer
// than 512 threads of `most` vectors hold.
struct NormPlan {
  int tpr = 0, vpt = 0, threads = 0;
};
NormPlan norm_plan(int64_t rows, int64_t nv, int most = 4) {
  NormPlan best;
  int64_t least = -1;
  const bool few = rows * nv < 512 * (int64_t)device_sms();
  for (int tpr = 8; tpr <= ssm::kNormMaxTpr; tpr *= 2)
    for (int vpt = 1; vpt <= most; ++vpt) {
      const int64_t idle = (int64_t)tpr * vpt - nv;
      if (idle < 0) continue;
      const int64_t cost = few ? vpt * (int64_t)65536 + tpr : idle;
      if (least < 0 || cost < least) {
        least = cost;
        best.tpr = tpr;
        best.vpt = vpt;
      }
    }
  best.threads = best.tpr > ssm::kNormThreads ? best.tpr : ssm::kNormThreads;
  return best;
}
// CTAs of `threads` threads that an SM holds of a kernel, at most four: the
// backward runs in one wave of them, each with a partial row of the parameters'
// gradients (per group).  Asked for the most shared memory a call of it takes, so
// that the answer, and with it the order of the sums, is the same for every call.
constexpr int kNormMaxCtas = 4;
constexpr int kNormMostSmem = ssm::kNormThreads * 4 * ssm::kNormBwdElems * 4;
template <auto Kernel> int norm_ctas(int threads) {
  static PerDevice ctas[2];
  return ctas[threads <= ssm::kNormThreads ? 0 : 1].get(
      [threads](int) {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, threads, kNormMostSmem) != cudaSuccess) {
          cudaGetLastError();
          n = 1;
        }
        return n < 1 ? 1 : n > kNormMaxCtas ? kNormMaxCtas : n;
      },
      1);
}
int64_t norm_parts(int64_t rows, int64_t groups, const NormPlan &n, int ctas) {
  const int64_t slots = n.threads / n.tpr;
  int64_t parts = ctas * (int64_t)device_sms() / groups;
  if (parts < 1) parts = 1;
  const int64_t rounds = (rows + parts * slots - 1) / (parts * slots);  // rows a slot takes
  return (rows + rounds * slots - 1) / (rounds * slots);
}
int64_t norm_bwd_parts(int64_t rows) {  // of whichever kernel
  const int64_t most = kNormMaxCtas * (int64_t)device_sms();
  return rows < most ? rows : most;
}

// Dynamic shared memory of a backward CTA: its slots' columns, summed at its end.
int norm_smem(const NormPlan &n, int64_t width) {
  const int64_t slots = n.threads / n.tpr;
  return slots > 1 ? (int)(slots * width * 4) : 0;
}

// f(integral_constant<int, vpt>) for 1 <= vpt <= MOST
template <int MOST, typename F> ssm_status by_vpt(int vpt, F &&f) {
  if constexpr (MOST > 1)
    if (vpt < MOST) return by_vpt<MOST - 1>(vpt, f);
  return f(std::integral_constant<int, MOST>());
}

template <typename T, int E, int FORM>
ssm_status gated_norm_fwd_e(ssm::GatedNormParams p, cudaStream_t st) {
  const char *what = "ssm_gated_norm_fwd";
  const int64_t rows = p.rows * p.groups;
  const NormPlan n = norm_plan(rows, p.d / p.groups / E);
  if (n.tpr == 0) {
    const unsigned grid = (unsigned)(rows < (1 << 20) ? rows : (1 << 20));
    ssm::gated_norm_fwd_long_kernel<T><<<grid, ssm::kNormThreads, 0, st>>>(p);
    return check_launch(what);
  }
  p.tpr = n.tpr;
  const int64_t slots = n.threads / n.tpr, blocks = (rows + slots - 1) / slots;
  if (blocks > kMaxGrid) return fail(SSM_ERR_UNSUPPORTED, "%s: too many rows for one grid", what);
  return by_vpt<4>(n.vpt, [&](auto vpt) {
    ssm::gated_norm_fwd_kernel<T, E, decltype(vpt)::value, FORM><<<(unsigned)blocks, n.threads, 0, st>>>(p);
    return check_launch(what);
  });
}
template <typename T, int E> ssm_status gated_norm_fwd_f(const ssm::GatedNormParams &p, cudaStream_t st) {
  if (!p.z) return gated_norm_fwd_e<T, E, ssm::kNoGate>(p, st);
  return p.before ? gated_norm_fwd_e<T, E, ssm::kNormFirst>(p, st)
                  : gated_norm_fwd_e<T, E, ssm::kGateFirst>(p, st);
}
template <typename T> ssm_status gated_norm_fwd_any(const ssm::GatedNormParams &p, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  if (vec_rows(E, sizeof(T), p.d / p.groups, {{p.x, p.x_ld}, {p.z, p.z_ld}, {p.y, p.y_ld}}) &&
      aligned(p.w, 16))
    return gated_norm_fwd_f<T, E>(p, st);
  return gated_norm_fwd_f<T, 1>(p, st);
}

template <typename T, int E, int FORM>
ssm_status gated_norm_bwd_e(ssm::GatedNormBwdParams q, int64_t *parts, cudaStream_t st) {
  const char *what = "ssm_gated_norm_bwd";
  ssm::GatedNormParams &p = q.f;
  const NormPlan n = norm_plan(p.rows * p.groups, p.d / p.groups / E);
  if (n.tpr == 0) {
    *parts = norm_bwd_parts(p.rows);
    ssm::gated_norm_bwd_long_kernel<T><<<(unsigned)*parts, ssm::kNormThreads, 0, st>>>(q);
    return check_launch(what);
  }
  p.tpr = n.tpr;
  const int smem = norm_smem(n, p.d / p.groups);
  return by_vpt<4>(n.vpt, [&](auto vpt) {
    constexpr auto kernel = ssm::gated_norm_bwd_kernel<T, E, decltype(vpt)::value, FORM>;
    *parts = norm_parts(p.rows, p.groups, n, norm_ctas<kernel>(n.threads));
    q.parts = (int)*parts;
    if (*parts > kMaxGrid / p.groups) return fail(SSM_ERR_UNSUPPORTED, "%s: too many groups", what);
    kernel<<<(unsigned)(*parts * p.groups), n.threads, smem, st>>>(q);
    return check_launch(what);
  });
}
template <typename T, int E>
ssm_status gated_norm_bwd_f(const ssm::GatedNormBwdParams &q, int64_t *parts, cudaStream_t st) {
  if (!q.f.z) return gated_norm_bwd_e<T, E, ssm::kNoGate>(q, parts, st);
  return q.f.before ? gated_norm_bwd_e<T, E, ssm::kNormFirst>(q, parts, st)
                    : gated_norm_bwd_e<T, E, ssm::kGateFirst>(q, parts, st);
}
template <typename T>
ssm_status gated_norm_bwd_any(const ssm::GatedNormBwdParams &q, int64_t *parts, cudaStream_t st) {
  constexpr int E = ssm::kNormBwdElems;
  const ssm::GatedNormParams &p = q.f;
  if (vec_rows(E, sizeof(T), p.d / p.groups,
               {{p.x, p.x_ld}, {p.z, p.z_ld}, {q.dy, q.dy_ld}, {q.dx, q.dx_ld}, {q.dz, q.dz_ld}}) &&
      aligned(p.w, 16))
    return gated_norm_bwd_f<T, E>(q, parts, st);
  return gated_norm_bwd_f<T, 1>(q, parts, st);
}

bool add_norm_vec(int64_t E, size_t es, size_t rs, const ssm::AddNormParams &p,
                  std::initializer_list<std::pair<const void *, int64_t>> act,
                  std::initializer_list<std::pair<const void *, int64_t>> res) {
  if (!vec_rows(E, es, p.d, act) || !aligned(p.w, 16)) return false;
  if (p.d % E != 0 || (p.post && !aligned(p.post, 16)) || (p.scale && !aligned(p.scale, 16))) return false;
  for (const auto &r : res) {  // at most 16 bytes an access
    const size_t a = E * rs < 16 ? E * rs : 16;
    if (r.first && (!aligned(r.first, a) || r.second * rs % a != 0)) return false;
  }
  return true;
}

template <typename T, typename R, int E>
ssm_status add_norm_fwd_e(ssm::AddNormParams p, cudaStream_t st) {
  const char *what = "ssm_add_norm_fwd";
  const NormPlan n = norm_plan(p.rows, p.d / E);
  if (n.tpr == 0) {
    const unsigned grid = (unsigned)(p.rows < (1 << 20) ? p.rows : (1 << 20));
    ssm::add_norm_fwd_long_kernel<T, R><<<grid, ssm::kNormThreads, 0, st>>>(p);
    return check_launch(what);
  }
  p.tpr = n.tpr;
  const int64_t slots = n.threads / n.tpr, blocks = (p.rows + slots - 1) / slots;
  if (blocks > kMaxGrid) return fail(SSM_ERR_UNSUPPORTED, "%s: too many rows for one grid", what);
  return by_vpt<4>(n.vpt, [&](auto vpt) {
    ssm::add_norm_fwd_kernel<T, R, E, decltype(vpt)::value><<<(unsigned)blocks, n.threads, 0, st>>>(p);
    return check_launch(what);
  });
}
template <typename T, typename R> ssm_status add_norm_fwd_any(const ssm::AddNormParams &p, cudaStream_t st) {
  constexpr int E = 16 / sizeof(T);
  if (add_norm_vec(E, sizeof(T), sizeof(R), p, {{p.x, p.x_ld}, {p.y, p.y_ld}},
                   {{p.res, p.res_ld}, {p.res_out, p.ro_ld}}))
    return add_norm_fwd_e<T, R, E>(p, st);
  return add_norm_fwd_e<T, R, 1>(p, st);
}

template <typename T, typename R, int E, bool POST, bool SCALE>
ssm_status add_norm_bwd_f(ssm::AddNormBwdParams q, int64_t *parts, cudaStream_t st) {
  const char *what = "ssm_add_norm_bwd";
  // with x and its sums at most two vectors a thread, where that leaves no more
  // than a quarter of the threads idle, else three: more spill (bf16, 16384 x 768,
  // scale and post norm: 2 a thread 62 us, 3 73)
  const int64_t nv = q.f.d / E;
  NormPlan n = norm_plan(q.f.rows, nv, POST || SCALE ? 2 : 4);
  if ((POST || SCALE) && (n.tpr == 0 || 3 * (int64_t)n.tpr * n.vpt > 4 * nv))
    n = norm_plan(q.f.rows, nv, 3);
  if (n.tpr == 0) {
    *parts = norm_bwd_parts(q.f.rows);
    ssm::add_norm_bwd_long_kernel<T, R><<<(unsigned)*parts, ssm::kNormThreads, 0, st>>>(q);
    return check_launch(what);
  }
  q.f.tpr = n.tpr;
  const int smem = norm_smem(n, q.f.d);
  return by_vpt<POST || SCALE ? 3 : 4>(n.vpt, [&](auto vpt) {
    constexpr auto kernel = ssm::add_norm_bwd_kernel<T, R, E, decltype(vpt)::value, POST, SCALE>;
    *parts = norm_parts(q.f.rows, 1, n, norm_ctas<kernel>(n.threads));
    q.parts = (int)*parts;
    kernel<<<(unsigned)*parts, n.threads, smem, st>>>(q);
    return check_launch(what);
  });
}
template <typename T, typename R, int E>
ssm_status add_norm_bwd_e(const ssm::AddNormBwdParams &q, int64_t *parts, cudaStream_t st) {
  if (q.f.post)
    return q.f.scale ? add_norm_bwd_f<T, R, E, true, true>(q, parts, st)
                     : add_norm_bwd_f<T, R, E, true, false>(q, parts, st);
  return q.f.scale ? add_norm_bwd_f<T, R, E, false, true>(q, parts, st)
                   : add_norm_bwd_f<T, R, E, false, false>(q, parts, st);
}
template <typename T, typename R>
ssm_status add_norm_bwd_any(const ssm::AddNormBwdParams &q, int64_t *parts, cudaStream_t st) {
  constexpr int E = ssm::kNormBwdElems;
  if (add_norm_vec(E, sizeof(T), sizeof(R), q.f, {{q.f.x, q.f.x_ld}, {q.dy, q.dy_ld}, {q.dx, q.dx_ld}},
                   {{q.f.res_out, q.f.ro_ld}, {q.dro, q.dro_ld}, {q.dres, q.dres_ld}}))
    return add_norm_bwd_e<T, R, E>(q, parts, st);
  return add_norm_bwd_e<T, R, 1>(q, parts, st);
}

ssm_status check_eps(const char *what, float eps) {
  return std::isfinite(eps) && eps >= 0.0f
             ? SSM_OK
             : fail(SSM_ERR_INVALID_ARG, "%s: eps is negative or not finite", what);
}

ssm_status check_gated_norm(const char *what, Args &a, const ssm::GatedNormParams &p,
                            ssm_dtype dtype) {
  if (ssm_status s = bad_dtype(what, dtype)) return s;
  if (!sizes_ok({p.rows, p.d}))
    return fail(SSM_ERR_INVALID_ARG, "%s: negative size or sizes that overflow int64", what);
  if (p.groups < 1 || p.d % p.groups != 0)
    return fail(SSM_ERR_INVALID_ARG, "%s: groups %lld does not divide d %lld", what,
                (long long)p.groups, (long long)p.d);
  if (ssm_status s = check_eps(what, p.eps)) return s;
  if (p.rows > 0 && p.d > 0 && (!p.x || !p.w))
    return fail(SSM_ERR_INVALID_ARG, "%s: x and weight are required", what);
  a.rows(false, "x", p.x, p.rows, p.d, p.x_ld);
  a.rows(false, "z", p.z, p.rows, p.d, p.z_ld);
  a.flat(false, "weight", p.w, p.d * 4);
  return SSM_OK;
}

ssm_status check_add_norm(const char *what, Args &a, const ssm::AddNormParams &p, ssm_dtype dtype,
                          ssm_dtype rdtype) {
  if (ssm_status s = bad_dtype(what, dtype)) return s;
  if (rdtype != SSM_F32 && rdtype != dtype)
    return fail(SSM_ERR_UNSUPPORTED, "%s: residual_dtype %d is neither SSM_F32 nor dtype", what,
                (int)rdtype);
  if (!sizes_ok({p.rows, p.d, 3}))
    return fail(SSM_ERR_INVALID_ARG, "%s: negative size or sizes that overflow int64", what);
  if (ssm_status s = check_eps(what, p.eps)) return s;
  if (p.rows > 0 && p.d > 0 && !p.w) return fail(SSM_ERR_INVALID_ARG, "%s: weight is required", what);
  a.rows(false, "x", p.x, p.rows, p.d, p.x_ld);
  a.flat(false, "weight", p.w, p.d * 4);
  a.flat(false, "post_weight", p.post, p.d * 4);
  a.flat(false, "scale", p.scale, p.d * 4);
  return SSM_OK;
}

}  // namespace

#ifdef SSM_DEBUG_BOUNDS
cudaError_t ssm_host::take_block_bounds_word(unsigned int *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_ssm_bounds_word, sizeof *word);
  if (e == cudaSuccess && *word) {
    const unsigned int none = 0;
    e = cudaMemcpyToSymbol(g_ssm_bounds_word, &none, sizeof none);
  }
  return e;
}
#endif

extern "C" {

size_t ssm_gated_scan_states_bytes(int64_t b, int64_t L, int64_t d_in) {
  if (!sizes_ok({b, L, d_in})) return (size_t)-1;
  return (size_t)(b * gated_chunks(L) * d_in) * 4;
}

ssm_status ssm_gated_scan_fwd(const void *u, int64_t u_ld, const void *gate_a, int64_t gate_a_ld,
                              const void *gate_x, int64_t gate_x_ld, const float *A,
                              const float *bias_a, const float *bias_x, const void *z,
                              int64_t z_ld, const uint8_t *seq_start, const float *h0,
                              float *h_last, void *y, int64_t y_ld, float *chunk_states,
                              size_t chunk_states_bytes, int64_t b, int64_t L, int64_t d_in,
                              ssm_dtype dtype, ssm_stream_t stream) {
  const char *what = "ssm_gated_scan_fwd";
  g_last_error.clear();
  ssm::GatedParams p{u, gate_a, gate_x, z, ld32(u_ld), ld32(gate_a_ld), ld32(gate_x_ld), ld32(z_ld), A,
                     bias_a, bias_x, seq_start, h0, h_last, y, ld32(y_ld), chunk_states, b, L, d_in};
  Args a(what, esize(dtype));
  if (ssm_status s = check_gated(what, a, p, dtype)) return s;
  if (b * L > 0 && d_in > 0 && !y) return fail(SSM_ERR_INVALID_ARG, "%s: y is required", what);
  a.flat(false, "h0", h0, b * d_in * 4);
  a.flat(true, "h_last", h_last, b * d_in * 4);
  a.rows(true, "y", y, b * L, d_in, y_ld);
  a.flat(true, "chunk_states", chunk_states, b * gated_chunks(L) * d_in * 4);
  a.same("h_last", "h0");
  if (ssm_status s = a.check()) return s;
  if (chunk_states)
    if (ssm_status s = check_states(what, chunk_states, chunk_states_bytes, b, L, d_in)) return s;
  if (b == 0 || d_in == 0) return ok();
  if (L == 0) return pass_state(h0, h_last, b * d_in, cu(stream), what);
  return dtype == SSM_BF16 ? gated_fwd_any<__nv_bfloat16>(p, cu(stream))
                           : gated_fwd_any<float>(p, cu(stream));
}

size_t ssm_gated_scan_bwd_workspace_bytes(int64_t b, int64_t L, int64_t d_in) {
  if (!sizes_ok({b, L, d_in, 3})) return (size_t)-1;
  return (size_t)(gated_bwd_parts(b, L, d_in) * 3 * d_in) * 4;
}

ssm_status ssm_gated_scan_bwd(const void *u, int64_t u_ld, const void *gate_a, int64_t gate_a_ld,
                              const void *gate_x, int64_t gate_x_ld, const float *A,
                              const float *bias_a, const float *bias_x, const void *z,
                              int64_t z_ld, const uint8_t *seq_start, const void *dout,
                              int64_t dout_ld, const float *dh_last, void *du, int64_t du_ld,
                              void *dgate_a, int64_t dgate_a_ld, void *dgate_x,
                              int64_t dgate_x_ld, void *dz, int64_t dz_ld, float *dA,
                              float *dbias_a, float *dbias_x, float *dh0, int64_t b, int64_t L,
                              int64_t d_in, ssm_dtype dtype, const float *chunk_states,
                              size_t chunk_states_bytes, void *workspace, size_t workspace_bytes,
                              ssm_stream_t stream) {
  const char *what = "ssm_gated_scan_bwd";
  g_last_error.clear();
  if (!z) dz = nullptr;
  ssm::GatedParams f{u, gate_a, gate_x, z, ld32(u_ld), ld32(gate_a_ld), ld32(gate_x_ld), ld32(z_ld), A,
                     bias_a, bias_x, seq_start, nullptr, nullptr, nullptr, 0,
                     const_cast<float *>(chunk_states), b, L, d_in};
  Args a(what, esize(dtype));
  if (ssm_status s = check_gated(what, a, f, dtype)) return s;
  const int64_t R = b * L;
  if (R > 0 && d_in > 0 && (!dout || !du || !dgate_a || !dgate_x || !chunk_states || (z && !dz)))
    return fail(SSM_ERR_INVALID_ARG, "%s: dout, du, dgate_a, dgate_x, chunk_states and, with z, dz "
                "are required", what);
  if (d_in > 0 && !dA) return fail(SSM_ERR_INVALID_ARG, "%s: dA is required", what);
  const size_t need = ssm_gated_scan_bwd_workspace_bytes(b, L, d_in);
  a.rows(false, "dout", dout, R, d_in, dout_ld);
  a.flat(false, "dh_last", dh_last, b * d_in * 4);
  a.flat(false, "chunk_states", chunk_states, b * gated_chunks(L) * d_in * 4);
  a.rows(true, "du", du, R, d_in, du_ld);
  a.rows(true, "dgate_a", dgate_a, R, d_in, dgate_a_ld);
  a.rows(true, "dgate_x", dgate_x, R, d_in, dgate_x_ld);
  a.rows(true, "dz", dz, R, d_in, dz_ld);
  a.flat(true, "dA", dA, d_in * 4);
  a.flat(true, "dbias_a", dbias_a, d_in * 4);
  a.flat(true, "dbias_x", dbias_x, d_in * 4);
  a.flat(true, "dh0", dh0, b * d_in * 4);
  a.flat(true, "workspace", workspace, (int64_t)need, 16);
  a.same("dh0", "dh_last");
  if (ssm_status s = a.check()) return s;
  const cudaStream_t st = cu(stream);
  if (d_in == 0) return ok();
  if (R == 0) {
    for (float *g : {dA, dbias_a, dbias_x})
      if (ssm_status s = zero(g, d_in, st, what)) return s;
    return pass_state(dh_last, dh0, b * d_in, st, what);
  }
  if (ssm_status s = check_states(what, chunk_states, chunk_states_bytes, b, L, d_in)) return s;
  if (ssm_status s = need_workspace(what, workspace, workspace_bytes, need)) return s;
  float *part = static_cast<float *>(workspace);
  ssm::GatedBwdParams q{f,  dout, ld32(dout_ld), dh_last, du, dgate_a, dgate_x, dz, ld32(du_ld),
                        ld32(dgate_a_ld), ld32(dgate_x_ld), ld32(dz_ld), dh0, part};
  int64_t parts = 0;
  if (ssm_status s = dtype == SSM_BF16 ? gated_bwd_any<__nv_bfloat16>(q, &parts, st)
                                       : gated_bwd_any<float>(q, &parts, st))
    return s;
  return col_sum(part, parts, d_in, dA, d_in, dbias_a, d_in, dbias_x, st, what);
}

ssm_status ssm_gated_state_update(float *state, const void *u, int64_t u_ld, const void *gate_a,
                                  int64_t gate_a_ld, const void *gate_x, int64_t gate_x_ld,
                                  const float *A, const float *bias_a, const float *bias_x,
                                  const void *z, int64_t z_ld, void *y, int64_t y_ld, int64_t b,
                                  int64_t d_in, ssm_dtype dtype, ssm_stream_t stream) {
  const char *what = "ssm_gated_state_update";
  g_last_error.clear();
  ssm::GatedParams p{u, gate_a, gate_x, z, ld32(u_ld), ld32(gate_a_ld), ld32(gate_x_ld), ld32(z_ld), A,
                     bias_a, bias_x, nullptr, nullptr, nullptr, y, ld32(y_ld), nullptr, b, 1, d_in};
  Args a(what, esize(dtype));
  if (ssm_status s = check_gated(what, a, p, dtype)) return s;
  if (b > 0 && d_in > 0 && (!state || !y))
    return fail(SSM_ERR_INVALID_ARG, "%s: state and y are required", what);
  a.flat(true, "state", state, b * d_in * 4);
  a.rows(true, "y", y, b, d_in, y_ld);
  if (ssm_status s = a.check()) return s;
  if (b == 0 || d_in == 0) return ok();
  return dtype == SSM_BF16 ? gated_step_any<__nv_bfloat16>(p, state, cu(stream))
                           : gated_step_any<float>(p, state, cu(stream));
}

ssm_status ssm_conv1d_fwd(const void *x, int64_t x_ld, const float *weight, const float *bias,
                          int silu, const void *conv_state, void *conv_state_out,
                          const uint8_t *seq_start, void *y, int64_t y_ld, int64_t b, int64_t L,
                          int64_t d_in, int64_t d_conv, ssm_dtype dtype, ssm_stream_t stream) {
  const char *what = "ssm_conv1d_fwd";
  g_last_error.clear();
  ssm::ConvParams p{x, x_ld, weight, bias, silu != 0, conv_state, conv_state_out, seq_start, y, y_ld,
                    b, L, d_in};
  Args a(what, esize(dtype));
  if (ssm_status s = check_conv(what, a, p, d_conv, dtype)) return s;
  if (b * L > 0 && d_in > 0 && !y) return fail(SSM_ERR_INVALID_ARG, "%s: y is required", what);
  // the kernel that writes the window takes its taps first, of an empty sequence too
  if (b > 0 && d_in > 0 && conv_state_out && !weight)
    return fail(SSM_ERR_INVALID_ARG, "%s: weight is required", what);
  const size_t es = esize(dtype);
  a.flat(false, "conv_state", conv_state, b * d_in * d_conv * (int64_t)es, es);
  a.flat(true, "conv_state_out", conv_state_out, b * d_in * d_conv * (int64_t)es, es);
  a.rows(true, "y", y, b * L, d_in, y_ld);
  a.same("conv_state_out", "conv_state");
  if (ssm_status s = a.check()) return s;
  if (b == 0 || d_in == 0 || (L == 0 && !conv_state_out)) return ok();
  return conv_dispatch(dtype, d_conv, [&](auto t, auto k) {
    return conv_fwd_k<decltype(t), decltype(k)::value>(p, cu(stream));
  });
}

size_t ssm_conv1d_bwd_workspace_bytes(int64_t b, int64_t L, int64_t d_in, int64_t d_conv) {
  if (d_conv < 1 || d_conv > ssm::kMaxConv || !sizes_ok({b, L, d_in, d_conv + 1})) return (size_t)-1;
  return (size_t)(conv_bwd_parts(b, L, d_in) * d_in * (d_conv + 1)) * 4;
}

ssm_status ssm_conv1d_bwd(const void *x, int64_t x_ld, const float *weight, const float *bias,
                          int silu, const void *conv_state, const uint8_t *seq_start,
                          const void *dy, int64_t dy_ld, void *dx, int64_t dx_ld, float *dweight,
                          float *dbias, int64_t b, int64_t L, int64_t d_in, int64_t d_conv,
                          ssm_dtype dtype, void *workspace, size_t workspace_bytes,
                          ssm_stream_t stream) {
  const char *what = "ssm_conv1d_bwd";
  g_last_error.clear();
  ssm::ConvParams p{x, x_ld, weight, bias, silu != 0, conv_state, nullptr, seq_start, nullptr, 0, b, L,
                    d_in};
  Args a(what, esize(dtype));
  if (ssm_status s = check_conv(what, a, p, d_conv, dtype)) return s;
  const int64_t R = b * L;
  if (R > 0 && d_in > 0 && (!dy || !dx))
    return fail(SSM_ERR_INVALID_ARG, "%s: dy and dx are required", what);
  if (d_in > 0 && !dweight) return fail(SSM_ERR_INVALID_ARG, "%s: dweight is required", what);
  const size_t es = esize(dtype), need = ssm_conv1d_bwd_workspace_bytes(b, L, d_in, d_conv);
  a.flat(false, "conv_state", conv_state, b * d_in * d_conv * (int64_t)es, es);
  a.rows(false, "dy", dy, R, d_in, dy_ld);
  a.rows(true, "dx", dx, R, d_in, dx_ld);
  a.flat(true, "dweight", dweight, d_in * d_conv * 4);
  a.flat(true, "dbias", dbias, d_in * 4);
  a.flat(true, "workspace", workspace, (int64_t)need, 16);
  if (ssm_status s = a.check()) return s;
  const cudaStream_t st = cu(stream);
  if (d_in == 0) return ok();
  if (R == 0) {
    if (ssm_status s = zero(dweight, d_in * d_conv, st, what)) return s;
    return zero(dbias, d_in, st, what);
  }
  if (ssm_status s = need_workspace(what, workspace, workspace_bytes, need)) return s;
  float *part = static_cast<float *>(workspace);
  ssm::ConvBwdParams q{p, dy, dy_ld, dx, dx_ld, 0, part};
  int64_t parts = 0;
  if (ssm_status s = conv_dispatch(dtype, d_conv, [&](auto t, auto k) {
        return conv_bwd_k<decltype(t), decltype(k)::value>(q, &parts, st);
      }))
    return s;
  return col_sum(part, parts, d_in * d_conv, dweight, d_in, dbias, 0, nullptr, st,
                 what);
}

ssm_status ssm_conv1d_update(void *conv_state, const void *x, int64_t x_ld, const float *weight,
                             const float *bias, int silu, void *y, int64_t y_ld, int64_t b,
                             int64_t d_in, int64_t d_conv, ssm_dtype dtype, ssm_stream_t stream) {
  const char *what = "ssm_conv1d_update";
  g_last_error.clear();
  ssm::ConvParams p{x, x_ld, weight, bias, silu != 0, nullptr, nullptr, nullptr, y, y_ld, b, 1, d_in};
  Args a(what, esize(dtype));
  if (ssm_status s = check_conv(what, a, p, d_conv, dtype)) return s;
  if (b > 0 && d_in > 0 && (!conv_state || !y))
    return fail(SSM_ERR_INVALID_ARG, "%s: conv_state and y are required", what);
  const size_t es = esize(dtype);
  a.flat(true, "conv_state", conv_state, b * d_in * d_conv * (int64_t)es, es);
  a.rows(true, "y", y, b, d_in, y_ld);
  if (ssm_status s = a.check()) return s;
  if (b == 0 || d_in == 0) return ok();
  return conv_dispatch(dtype, d_conv, [&](auto t, auto k) {
    return conv_step_k<decltype(t), decltype(k)::value>(p, conv_state, cu(stream));
  });
}

ssm_status ssm_gated_norm_fwd(const void *x, int64_t x_ld, const void *z, int64_t z_ld,
                              const float *weight, int64_t groups, float eps,
                              int norm_before_gate, void *y, int64_t y_ld, int64_t rows, int64_t d,
                              ssm_dtype dtype, ssm_stream_t stream) {
  const char *what = "ssm_gated_norm_fwd";
  g_last_error.clear();
  ssm::GatedNormParams p{x, z, x_ld, z_ld, weight, groups, eps, norm_before_gate != 0, y, y_ld, rows, d};
  Args a(what, esize(dtype));
  if (ssm_status s = check_gated_norm(what, a, p, dtype)) return s;
  if (rows > 0 && d > 0 && !y) return fail(SSM_ERR_INVALID_ARG, "%s: y is required", what);
  a.rows(true, "y", y, rows, d, y_ld);
  if (ssm_status s = a.check()) return s;
  if (rows == 0 || d == 0) return ok();
  return dtype == SSM_BF16 ? gated_norm_fwd_any<__nv_bfloat16>(p, cu(stream))
                           : gated_norm_fwd_any<float>(p, cu(stream));
}

size_t ssm_gated_norm_bwd_workspace_bytes(int64_t rows, int64_t d, int64_t groups) {
  if (groups < 1 || !sizes_ok({rows, d}) || d % groups != 0) return (size_t)-1;
  return (size_t)(norm_bwd_parts(rows) * d) * 4;
}

ssm_status ssm_gated_norm_bwd(const void *x, int64_t x_ld, const void *z, int64_t z_ld,
                              const float *weight, int64_t groups, float eps,
                              int norm_before_gate, const void *dy, int64_t dy_ld, void *dx,
                              int64_t dx_ld, void *dz, int64_t dz_ld, float *dweight, int64_t rows,
                              int64_t d, ssm_dtype dtype, void *workspace, size_t workspace_bytes,
                              ssm_stream_t stream) {
  const char *what = "ssm_gated_norm_bwd";
  g_last_error.clear();
  if (!z) dz = nullptr;
  ssm::GatedNormParams p{x, z, x_ld, z_ld, weight, groups, eps, norm_before_gate != 0, nullptr, 0, rows, d};
  Args a(what, esize(dtype));
  if (ssm_status s = check_gated_norm(what, a, p, dtype)) return s;
  if (rows > 0 && d > 0 && (!dy || !dx || (z && !dz)))
    return fail(SSM_ERR_INVALID_ARG, "%s: dy, dx and, with z, dz are required", what);
  if (d > 0 && !dweight) return fail(SSM_ERR_INVALID_ARG, "%s: dweight is required", what);
  const size_t need = ssm_gated_norm_bwd_workspace_bytes(rows, d, groups);
  a.rows(false, "dy", dy, rows, d, dy_ld);
  a.rows(true, "dx", dx, rows, d, dx_ld);
  a.rows(true, "dz", dz, rows, d, dz_ld);
  a.flat(true, "dweight", dweight, d * 4);
  a.flat(true, "workspace", workspace, (int64_t)need, 16);
  if (ssm_status s = a.check()) return s;
  const cudaStream_t st = cu(stream);
  if (d == 0) return ok();
  if (rows == 0) return zero(dweight, d, st, what);
  if (ssm_status s = need_workspace(what, workspace, workspace_bytes, need)) return s;
  float *part = static_cast<float *>(workspace);
  ssm::GatedNormBwdParams q{p, dy, dy_ld, dx, dz, dx_ld, dz_ld, 0, part};
  int64_t n = 0;
  if (ssm_status s = dtype == SSM_BF16 ? gated_norm_bwd_any<__nv_bfloat16>(q, &n, st)
                                       : gated_norm_bwd_any<float>(q, &n, st))
    return s;
  return col_sum(part, n, d, dweight, 0, nullptr, 0, nullptr, st, what);
}

ssm_status ssm_add_norm_fwd(const void *x, int64_t x_ld, const void *residual, int64_t residual_ld,
                            const float *weight, const float *post_weight, const float *scale,
                            float eps, void *y, int64_t y_ld, void *residual_out,
                            int64_t residual_out_ld, int64_t rows, int64_t d, ssm_dtype dtype,
                            ssm_dtype residual_dtype, ssm_stream_t stream) {
  const char *what = "ssm_add_norm_fwd";
  g_last_error.clear();
  ssm::AddNormParams p{x, residual, x_ld, residual_ld, weight, post_weight, scale, eps, y, residual_out,
                       y_ld, residual_out_ld, rows, d};
  Args a(what, esize(dtype));
  if (ssm_status s = check_add_norm(what, a, p, dtype, residual_dtype)) return s;
  if (rows > 0 && d > 0 && (!x || !y || !residual_out))
    return fail(SSM_ERR_INVALID_ARG, "%s: x, y and residual_out are required", what);
  a.rows(false, "residual", residual, rows, d, residual_ld, esize(residual_dtype));
  a.rows(true, "y", y, rows, d, y_ld);
  a.rows(true, "residual_out", residual_out, rows, d, residual_out_ld, esize(residual_dtype));
  a.same("residual_out", "residual");
  if (ssm_status s = a.check()) return s;
  if (rows == 0 || d == 0) return ok();
  using bf16 = __nv_bfloat16;
  if (dtype == SSM_F32) return add_norm_fwd_any<float, float>(p, cu(stream));
  return residual_dtype == SSM_F32 ? add_norm_fwd_any<bf16, float>(p, cu(stream))
                                   : add_norm_fwd_any<bf16, bf16>(p, cu(stream));
}

size_t ssm_add_norm_bwd_workspace_bytes(int64_t rows, int64_t d) {
  if (!sizes_ok({rows, d, 3})) return (size_t)-1;
  return (size_t)(norm_bwd_parts(rows) * 3 * d) * 4;
}

ssm_status ssm_add_norm_bwd(const void *x, int64_t x_ld, const void *residual_out,
                            int64_t residual_out_ld, const float *weight, const float *post_weight,
                            const float *scale, float eps, const void *dy, int64_t dy_ld,
                            const void *dresidual_out, int64_t dresidual_out_ld, void *dx,
                            int64_t dx_ld, void *dresidual, int64_t dresidual_ld, float *dweight,
                            float *dpost_weight, float *dscale, int64_t rows, int64_t d,
                            ssm_dtype dtype, ssm_dtype residual_dtype, void *workspace,
                            size_t workspace_bytes, ssm_stream_t stream) {
  const char *what = "ssm_add_norm_bwd";
  g_last_error.clear();
  if (!post_weight) dpost_weight = nullptr;
  if (!scale) dscale = nullptr;
  if (!post_weight && !scale) x = nullptr;
  ssm::AddNormParams p{x, nullptr, x_ld, 0, weight, post_weight, scale, eps, nullptr,
                       const_cast<void *>(residual_out), 0, residual_out_ld, rows, d};
  Args a(what, esize(dtype));
  if (ssm_status s = check_add_norm(what, a, p, dtype, residual_dtype)) return s;
  if (rows > 0 && d > 0 && (!residual_out || !dy || !dx || (!x && (post_weight || scale))))
    return fail(SSM_ERR_INVALID_ARG,
                "%s: residual_out, dy, dx and, with post_weight or scale, x are required", what);
  if (d > 0 && (!dweight || (post_weight && !dpost_weight) || (scale && !dscale)))
    return fail(SSM_ERR_INVALID_ARG,
                "%s: dweight and, with post_weight / scale, their gradients are required", what);
  const size_t rs = esize(residual_dtype), need = ssm_add_norm_bwd_workspace_bytes(rows, d);
  a.rows(false, "residual_out", residual_out, rows, d, residual_out_ld, rs);
  a.rows(false, "dy", dy, rows, d, dy_ld);
  a.rows(false, "dresidual_out", dresidual_out, rows, d, dresidual_out_ld, rs);
  a.rows(true, "dx", dx, rows, d, dx_ld);
  a.rows(true, "dresidual", dresidual, rows, d, dresidual_ld, rs);
  a.flat(true, "dweight", dweight, d * 4);
  a.flat(true, "dpost_weight", dpost_weight, d * 4);
  a.flat(true, "dscale", dscale, d * 4);
  a.flat(true, "workspace", workspace, (int64_t)need, 16);
  a.same("dresidual", "dresidual_out");
  if (ssm_status s = a.check()) return s;
  const cudaStream_t st = cu(stream);
  if (d == 0) return ok();
  if (rows == 0) {
    for (float *g : {dweight, dpost_weight, dscale})
      if (ssm_status s = zero(g, d, st, what)) return s;
    return ok();
  }
  if (ssm_status s = need_workspace(what, workspace, workspace_bytes, need)) return s;
  float *part = static_cast<float *>(workspace);
  ssm::AddNormBwdParams q{p, dy, dresidual_out, dy_ld, dresidual_out_ld, dx, dresidual, dx_ld,
                          dresidual_ld, 0, part};
  using bf16 = __nv_bfloat16;
  int64_t n = 0;
  if (ssm_status s = dtype == SSM_F32            ? add_norm_bwd_any<float, float>(q, &n, st)
                     : residual_dtype == SSM_F32 ? add_norm_bwd_any<bf16, float>(q, &n, st)
                                                 : add_norm_bwd_any<bf16, bf16>(q, &n, st))
    return s;
  return col_sum(part, n, d, dweight, d, dpost_weight, d, dscale, st, what);
}

}  // extern "C"
