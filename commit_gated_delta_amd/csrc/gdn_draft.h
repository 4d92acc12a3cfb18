// gdn_draft.h -- verification of drafted tokens against the model's
// probabilities from given random numbers, and the round's next token
// (gdn_draft_verify).  Compiled as part of gdn_state.hip.
//
// Row t of a lane's window gives the distribution p_t of the window's token
// t + 1, the drafter's row its own q_t (or the draft itself: q_t = 1 there).
// With w the drafted token it stands when u_t q_t(w) < p_t(w), so with the
// chance min(1, p / q).  The first draft that falls is replaced by a token
// of max(p_t - q_t, 0), and where all stand the last row gives one more: the
// tokens are then distributed as p says, whatever the drafter's q (Leviathan,
// Kalman & Matias, "Fast Inference from Transformers via Speculative
// Decoding", ICML 2023, Sec. 2.3 and appendix A.1).
//
// A token is where a running sum passes a given number, so an error d of the
// sums moves it with a chance of about d times the number of likely tokens:
// every exponential and sum here is f64.
#pragma once
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "gdn.h"
#include "gdn_scores.h"

namespace gdnv {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;
using gdnt::logit_at;
using gdnt::round16;
using gdnt::u32x4;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// What a slice of a row leaves behind: its largest logit (NaN if it holds
// one), the sum of 2^((x - m) c) with that as m, and the same without the
// row's draft.
struct Part {
  double z, zx;
  float m;
  int pad;
};

// What a lane's window comes to.
struct Verdict {
  int m;   // accepted prefix, the anchor included
  int ok;  // row m - 1 (and the drafter's, if a draft fell) has a distribution
  double top, z;              // of row m - 1
  double draft_top, draft_z;  // of the drafter's row m - 1, if a draft fell
};

struct DraftArgs {
  const void *logits, *draft;
  const int* tokens;
  const float* uniforms;
  const float* it;  // inverse temperature per lane
  int* m;
  int* next;
  float* accept;
  long stride, draft_stride;
  int lanes, t_max, vocab;
  int slices;        // of a row, in `parts`, from its first 16-byte line on
  int rest_slices;   // of a row, in `rest`, from its first id on
  Part* parts;       // [target rows, then drafter's rows][slices]
  double* rest;      // [lanes][rest_slices]: sums of max(p - q, 0)
  Verdict* verdicts;  // [lanes], of windows with drafts that have a distribution
};

constexpr int kSlice = 2048;   // ids of a slice
constexpr int kThreads = 256;  // of sum_kernel
constexpr int kWide = 1024;    // of the kernels behind it
constexpr int kRestSlices = 2;  // of a workgroup of rest_kernel

// 2^y for -1020 <= y <= 1, to 2e-14: a polynomial through the Chebyshev nodes
// of [-1/2, 1/2] for the fraction, the whole part added to the exponent.  (The
// library's exp takes twice the instructions.)
__device__ __forceinline__ double exp2_f64(double y) {
  constexpr double kWhole = 6755399441055744.0;  // 1.5 * 2^52: no fraction left
  const double t = y + kWhole, f = y - (t - kWhole);
  double e = 1.02059054137655955e-07;
  e = __builtin_fma(e, f, 1.32596452448871106e-06);
  e = __builtin_fma(e, f, 1.52526729248507372e-05);
  e = __builtin_fma(e, f, 1.54034337512510097e-04);
  e = __builtin_fma(e, f, 1.33335582007945925e-03);
  e = __builtin_fma(e, f, 9.61812919393431262e-03);
  e = __builtin_fma(e, f, 5.55041086646516704e-02);
  e = __builtin_fma(e, f, 2.40226506956403407e-01);
  e = __builtin_fma(e, f, 6.93147180559946174e-01);
  e = __builtin_fma(e, f, 1.00000000000001354e+00);
  u32x2 w = __builtin_bit_cast(u32x2, e);
  w[1] += __builtin_bit_cast(u32x2, t)[0] << 20;
  return __builtin_bit_cast(double, w);
}
// 2^((x - m) c), 0 below 2^-1000 (x = -inf among it).
constexpr double kLeast = -1000.0;
__device__ __forceinline__ double weight_of(float x, double m, double c) {
  const double y = ((double)x - m) * c;
  const double e = exp2_f64(__builtin_fmax(y, kLeast));
  return y >= kLeast ? e : 0.0;
}
// The same without the zeros, for sums in which 2^-1000 is nothing.
__device__ __forceinline__ double weight_in_sum(float x, double m, double c) {
  return exp2_f64(__builtin_fmax(((double)x - m) * c, kLeast));
}
// Sums of weights from which a slice counts: the largest of its 2^11 weights
// is then above 2^-1000, and so not 0 where an id is looked up.
constexpr double kNothing = 0x1p-950;
__device__ __forceinline__ double or_nothing(double sum) {
  return sum >= kNothing ? sum : 0.0;
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double x) {
  u32x2 w = __builtin_bit_cast(u32x2, x);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[i], CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, w);
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  u32x2 w = __builtin_bit_cast(u32x2, x);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)__builtin_amdgcn_readlane((int)w[i], lane);
  return __builtin_bit_cast(double, w);
}
// Sum over the 64 lanes, the same in every lane, in a fixed order.
__device__ __forceinline__ double wave_sum64(double x) {
  x += dpp64<0xB1>(x);
  x += dpp64<0x4E>(x);
  x += dpp64<0x141>(x);
  x += dpp64<0x140>(x);
  return (lane_value(x, 0) + lane_value(x, 16)) +
         (lane_value(x, 32) + lane_value(x, 48));
}
__device__ __forceinline__ double wave_scan64(double x) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 1; i < 64; i *= 2) {
    const double o = __shfl_up(x, i);
    if (lane >= i) x += o;
  }
  return x;
}
__device__ __forceinline__ float nan_max(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}
__device__ __forceinline__ float wave_nan_max(float x) {
  x = nan_max(x, gdn::dpp<0xB1>(x));
  x = nan_max(x, gdn::dpp<0x4E>(x));
  x = nan_max(x, gdn::dpp<0x141>(x));
  x = nan_max(x, gdn::dpp<0x140>(x));
  const int u = __float_as_int(x);
  return nan_max(nan_max(__int_as_float(__builtin_amdgcn_readlane(u, 0)),
                         __int_as_float(__builtin_amdgcn_readlane(u, 16))),
                 nan_max(__int_as_float(__builtin_amdgcn_readlane(u, 32)),
                         __int_as_float(__builtin_amdgcn_readlane(u, 48))));
}

// Inverse temperature of a lane times log2 e; 0: out of range.
__device__ __forceinline__ double exponent_of(const DraftArgs& p, int n) {
  const float it = p.it[n];
  return it >= 1e-30f && it <= 1e30f ? (double)it * 1.44269504088896340736 : 0.0;
}
template <typename T>
__device__ __forceinline__ const T* target_row(const DraftArgs& p, int n, int t) {
  return (const T*)p.logits + ((long)n * p.t_max + t) * p.stride;
}
template <typename T>
__device__ __forceinline__ const T* drafter_row(const DraftArgs& p, int n, int t) {
  return (const T*)p.draft + ((long)n * (p.t_max - 1) + t) * p.draft_stride;
}
// Logits of the row before its first 16-byte line starts (slices start there).
template <typename T>
__device__ __forceinline__ int skew_of(const T* x) {
  return (int)((uintptr_t)x % 16 / sizeof(T));
}

// One workgroup per G slices of a row, read once into registers.
template <typename T, int G>
__global__ __launch_bounds__(kThreads, 4) void sum_kernel(DraftArgs p,
                                                          gdn::LaneTable tl,
                                                          int groups) {
  constexpr int E = 16 / sizeof(T);              // logits per vector
  constexpr int VS = kSlice / (kThreads * E);    // vectors of a slice
  constexpr int V = G * VS;
  __shared__ float tops[4];
  __shared__ double sums[G][kThreads];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = blockIdx.x / groups, part = blockIdx.x % groups;
  const int targets = p.lanes * p.t_max;
  const bool drafter = row >= targets;
  const int per = drafter ? p.t_max - 1 : p.t_max;
  const int n = (drafter ? row - targets : row) / per;
  const int t = (drafter ? row - targets : row) % per;
  if (t >= tl.v[n] - (drafter ? 1 : 0)) return;
  const T* x = drafter ? drafter_row<T>(p, n, t) : target_row<T>(p, n, t);
  const int skew = skew_of(x);
  const u32x4* line = reinterpret_cast<const u32x4*>(x - skew);
  const int lines = (p.vocab + skew + E - 1) / E;
  const int first = part * kThreads * V + tid;

  u32x4 raw[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = first + k * kThreads;
    raw[k] = line[i < lines ? i : lines - 1];
  }
  // (only a row's draft without the drafter's distribution is left out)
  const int gone = !drafter && !p.draft && t + 1 < tl.v[n]
                       ? p.tokens[(long)n * p.t_max + t + 1]
                       : -1;
  const double c = exponent_of(p, n);
  float val[V][E];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = first + k * kThreads;
    const int id = i < lines ? i * E - skew : p.vocab;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (sizeof(T) == 4) val[k][e] = __uint_as_float(raw[k][e]);
      else
        val[k][e] = __uint_as_float(e & 1 ? raw[k][e / 2] & 0xffff0000u
                                          : raw[k][e / 2] << 16);
    }
    if (id < 0 || id > p.vocab - E) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((unsigned)(id + e) >= (unsigned)p.vocab) val[k][e] = -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) m = nan_max(m, val[k][e]);
  }
  m = wave_nan_max(m);
  if (lane == 0) tops[wave] = m;
  __syncthreads();
  m = nan_max(nan_max(tops[0], tops[1]), nan_max(tops[2], tops[3]));
  const double ref = m == -INFINITY ? 0.0 : (double)m;
  // the draft is taken out of its slice's sum, and added for a second one
  double own = 0.0;
  const int own_slice = gone < 0 || gone >= p.vocab ? -1 : (gone + skew) / kSlice;
  if (own_slice >= part * G && own_slice < (part + 1) * G) {
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((first + k * kThreads) * E - skew + e == gone) val[k][e] = -INFINITY;
    own = weight_of(logit_at(x, gone), ref, c);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    double z[2] = {0.0, 0.0};
#pragma unroll
    for (int k = 0; k < VS; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e)
        z[e & 1] += weight_in_sum(val[g * VS + k][e], ref, c);
    sums[g][tid] = z[0] + z[1];
  }
  __syncthreads();
  const int slice = part * G + wave;  // a wave adds one up
  if (wave >= G || slice >= p.slices) return;
  const double* of = sums[wave] + lane;
  const double zx =
      or_nothing(wave_sum64((of[0] + of[64]) + (of[128] + of[192])));
  if (lane == 0)
    p.parts[(long)row * p.slices + slice] = {
        slice == own_slice ? zx + own : zx, zx, m, 0};
}

// A workgroup of kWide threads works a lane's verdict out from the slices'
// sums, a wave a row.
struct Rows {
  float m[2][GDN_MAX_T];
  double z[2][GDN_MAX_T];
  int accepted;
};
template <typename T>
__device__ __forceinline__ Verdict decide(const DraftArgs& p, int n, int T_n,
                                          double c, Rows& rows, bool write) {
  const int lane = threadIdx.x & 63, wave = gdn::uniform(threadIdx.x >> 6);
  // the first wave's lanes hold a draft each: its logits are on their way
  // while the rows are summed up
  const bool drafted = wave == 0 && lane < T_n - 1;
  bool inside = false;
  float pw = 0.f, qw = 0.f, u = 0.f;
  if (drafted) {
    const int w = p.tokens[(long)n * p.t_max + lane + 1];
    u = p.uniforms[(long)n * p.t_max + lane];
    inside = (unsigned)w < (unsigned)p.vocab;
    const int i = inside ? w : 0;
    pw = logit_at(target_row<T>(p, n, lane), i);
    if (p.draft) qw = logit_at(drafter_row<T>(p, n, lane), i);
  }
  const int count = T_n + (p.draft ? T_n - 1 : 0);
  auto parts_of = [&](int r) {
    const long row = r < T_n ? (long)n * p.t_max + r
                             : (long)p.lanes * p.t_max +
                                   (long)n * (p.t_max - 1) + (r - T_n);
    return p.parts + row * p.slices;
  };
  constexpr int kStep = kWide / 64;
  const Part none = {0.0, 0.0, -INFINITY, 0};
  Part next = none;
  if (wave < count && lane < p.slices) next = parts_of(wave)[lane];
  for (int r = wave; r < count; r += kStep) {
    const Part* parts = parts_of(r);
    const Part first = next;
    next = none;
    if (r + kStep < count && lane < p.slices) next = parts_of(r + kStep)[lane];
    float m = first.m;
    for (int i = lane + 64; i < p.slices; i += 64) m = nan_max(m, parts[i].m);
    m = wave_nan_max(m);
    const double ref = m == -INFINITY ? 0.0 : (double)m;
    double z = first.z * weight_of(first.m, ref, c);
    for (int i = lane + 64; i < p.slices; i += 64)
      z += parts[i].z * weight_of(parts[i].m, ref, c);
    z = wave_sum64(z);
    if (lane == 0) {
      const int d = r >= T_n;
      rows.m[d][d ? r - T_n : r] = m;
      rows.z[d][d ? r - T_n : r] = z;
    }
  }
  __syncthreads();
  if (wave == 0) {
    bool stands = true;  // (lanes past the drafts)
    if (drafted) {
      const float m = rows.m[0][lane];
      bool ok = c > 0.0 && fabsf(m) < INFINITY;
      if (p.draft) ok = ok && fabsf(rows.m[1][lane]) < INFINITY;
      double a = 0.0, b = 1.0;  // chances of the draft
      if (ok && inside) {
        a = weight_of(pw, m, c) / rows.z[0][lane];
        if (p.draft) b = weight_of(qw, rows.m[1][lane], c) / rows.z[1][lane];
      }
      stands = ok && (double)u * b < a;
      if (write && p.accept)
        p.accept[(long)n * p.t_max + lane] =
            !ok ? NAN : a == 0.0 ? 0.f : a >= b ? 1.f : (float)(a / b);
    }
    const uint64_t fell = __ballot(!stands);
    if (lane == 0) rows.accepted = fell ? __builtin_ctzll(fell) + 1 : T_n;
  }
  __syncthreads();
  Verdict v;
  v.m = rows.accepted;
  const int t = v.m - 1;
  v.top = rows.m[0][t];
  v.z = rows.z[0][t];
  v.ok = c > 0.0 && fabsf(rows.m[0][t]) < INFINITY;
  v.draft_top = v.draft_z = 1.0;
  if (p.draft && v.m < T_n) {
    v.draft_top = rows.m[1][t];
    v.draft_z = rows.z[1][t];
    v.ok = v.ok && fabsf(rows.m[1][t]) < INFINITY;
  }
  return v;
}

// Weights of row m - 1 that the next token is taken by, apart from a common
// factor.
template <typename T>
struct Weights {
  const T *x, *y;  // the row and the drafter's, or NULL
  double top, draft_top, f, draft_f, c;
  int gone;        // an id of weight 0, or -1
  __device__ __forceinline__ double at(int i) const {
    double w = weight_of(logit_at(x, i), top, c) * f;
    if (y) {
      w -= weight_of(logit_at(y, i), draft_top, c) * draft_f;
      w = w > 0.0 ? w : 0.0;
    }
    return i == gone ? 0.0 : w;
  }
};
template <typename T>
__device__ __forceinline__ Weights<T> weights_of(const DraftArgs& p,
                                                 const Verdict& v, int n,
                                                 int T_n, double c, bool rest) {
  const int t = v.m - 1;
  Weights<T> w = {target_row<T>(p, n, t), nullptr, v.top, v.draft_top,
                  1.0 / v.z, 1.0 / v.draft_z, c, -1};
  if (rest && p.draft) w.y = drafter_row<T>(p, n, t);
  if (rest && !p.draft) w.gone = p.tokens[(long)n * p.t_max + t + 1];
  return w;
}

// With a drafter's distribution: the verdicts, and sums of max(p - q, 0) by
// slices of the row where a draft fell.
template <typename T>
__global__ __launch_bounds__(kWide) void rest_kernel(DraftArgs p,
                                                     gdn::LaneTable tl,
                                                     int groups) {
  __shared__ Rows rows;
  __shared__ double sums[kRestSlices][kWide / 64];
  const int n = blockIdx.x / groups, part = blockIdx.x % groups;
  const int T_n = tl.v[n], tid = threadIdx.x;
  if (T_n < 2) return;
  const double c = exponent_of(p, n);
  const Verdict v = decide<T>(p, n, T_n, c, rows, part == 0);
  if (part == 0 && tid == 0) p.verdicts[n] = v;
  if (!v.ok || v.m == T_n) return;
  const Weights<T> w = weights_of<T>(p, v, n, T_n, c, true);
#pragma unroll
  for (int g = 0; g < kRestSlices; ++g) {
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < kSlice / kWide; ++k) {
      const int i = (part * kRestSlices + g) * kSlice + k * kWide + tid;
      if (i < p.vocab) sum += w.at(i);
    }
    sum = wave_sum64(sum);
    if (tid % 64 == 0) sums[g][tid / 64] = sum;
  }
  __syncthreads();
  const int slice = part * kRestSlices + tid;
  if (tid >= kRestSlices || slice >= p.rest_slices) return;
  double sum = sums[tid][0];
  for (int i = 1; i < kWide / 64; ++i) sum += sums[tid][i];
  p.rest[(long)n * p.rest_slices + slice] = sum;
}

// The next token (and the verdict, where it is not there yet), a workgroup per
// lane: the slice that the border lies in, then the id within it.
template <typename T>
__global__ __launch_bounds__(kWide) void pick_kernel(DraftArgs p,
                                                     gdn::LaneTable tl) {
  __shared__ Rows rows;
  __shared__ double sums[kWide / 64];
  __shared__ double found[2];  // the running sum before the slice, and the border
  __shared__ int which, first_id[kWide / 64], last_id[kWide / 64];
  const int n = blockIdx.x, T_n = tl.v[n];
  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  if (T_n == 0) return;
  const double c = exponent_of(p, n);
  const Verdict v = p.draft && T_n > 1 ? p.verdicts[n]
                                       : decide<T>(p, n, T_n, c, rows, true);
  if (!v.ok) {
    if (tid == 0) {
      p.m[n] = v.m;
      p.next[n] = -1;
    }
    return;
  }
  bool rest = v.m < T_n;
  const int t = v.m - 1;
  const Part* parts = p.parts + ((long)n * p.t_max + t) * p.slices;
  const float u = p.uniforms[(long)n * p.t_max + T_n - 1];
  if (wave == 0) {
    const double share = u > 0.f ? u < 1.f ? (double)u : 1.0 : 0.0;
    auto slice_sum = [&](int i, int count) {
      if (i >= count) return 0.0;
      if (rest && p.draft) return p.rest[(long)n * p.rest_slices + i];
      return or_nothing((rest ? parts[i].zx : parts[i].z) *
                        weight_of(parts[i].m, v.top, c)) / v.z;
    };
    for (;;) {
      const int count = rest && p.draft ? p.rest_slices : p.slices;
      double whole = 0.0;
      for (int i0 = 0; i0 < count; i0 += 64)
        whole += lane_value(wave_scan64(slice_sum(i0 + lane, count)), 63);
      if (whole == 0.0 && rest) {  // nothing is left: from p
        rest = false;
        continue;
      }
      const double border = share * whole;
      double before = 0.0, base = 0.0;
      int got = -1, last = 0;
      double last_base = 0.0;
      for (int i0 = 0; i0 < count && got < 0; i0 += 64) {
        const double x = slice_sum(i0 + lane, count);
        const double upto = wave_scan64(x);
        const uint64_t hit = __ballot(before + upto > border && x > 0.0);
        const uint64_t some = __ballot(x > 0.0);
        if (hit) {
          const int l = __builtin_ctzll(hit);
          got = i0 + l;
          base = before + (l > 0 ? lane_value(upto, l - 1) : 0.0);
        }
        if (some) {
          const int l = 63 - __builtin_clzll(some);
          last = i0 + l;
          last_base = before + (l > 0 ? lane_value(upto, l - 1) : 0.0);
        }
        before += lane_value(upto, 63);
      }
      if (lane == 0) {
        which = (got >= 0 ? got : last) << 1 | (rest ? 1 : 0);
        found[0] = got >= 0 ? base : last_base;
        found[1] = border;
      }
      break;
    }
  }
  __syncthreads();
  rest = which & 1;
  const int slice = which >> 1;
  const Weights<T> w = weights_of<T>(p, v, n, T_n, c, rest);
  // ids of the slice, consecutive ones a thread
  constexpr int kPer = kSlice / kWide;
  const int skew = rest && p.draft ? 0 : skew_of(w.x);
  const int from = slice * kSlice - skew + tid * kPer;
  double mine = 0.0;
  double x[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = from + k;
    x[k] = (unsigned)i < (unsigned)p.vocab ? w.at(i) : 0.0;
    mine += x[k];
  }
  const double upto = wave_scan64(mine);
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  double run = found[0];
  for (int i = 0; i < wave; ++i) run += sums[i];
  const double below = __shfl_up(upto, 1);
  double at = lane > 0 ? run + below : run;
  int first = -1, last = -1;  // past the border; of any weight
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    at += x[k];
    if (x[k] > 0.0) {
      if (at > found[1] && first < 0) first = from + k;
      last = from + k;
    }
  }
  const uint64_t hit = __ballot(first >= 0), some = __ballot(last >= 0);
  // (the ids of a wave follow one another)
  const int by_first = hit ? __shfl(first, __builtin_ctzll(hit)) : -1;
  const int by_last = some ? __shfl(last, 63 - __builtin_clzll(some)) : -1;
  if (lane == 0) {
    first_id[wave] = by_first;
    last_id[wave] = by_last;
  }
  __syncthreads();
  if (tid != 0) return;
  int token = -1;
  for (int i = 0; i < kWide / 64 && token < 0; ++i) token = first_id[i];
  for (int i = kWide / 64 - 1; i >= 0 && token < 0; --i) token = last_id[i];
  p.m[n] = v.m;
  p.next[n] = token;
}

// ---------------------------------------------------------------- host side
static bool sizes_ok(int32_t n_lanes, int32_t t_max, int32_t vocab) {
  return n_lanes >= 1 && n_lanes <= GDN_MAX_LANES && t_max >= 1 &&
         t_max <= GDN_MAX_T && vocab >= 1 && vocab <= 1 << 30;
}
static int slices_for(int32_t vocab) { return (vocab + kSlice - 1) / kSlice; }
static size_t bytes_for(int32_t n_lanes, int32_t t_max, int32_t vocab,
                        int slices) {
  return round16((size_t)n_lanes * (2 * t_max - 1) * slices * sizeof(Part)) +
         round16((size_t)n_lanes * slices_for(vocab) * sizeof(double)) +
         round16((size_t)n_lanes * sizeof(Verdict));
}

// Four slices a workgroup (8 logits a thread each), or one where that would
// leave most of the CUs without any.
template <typename T>
static hipError_t run(const DraftArgs& p, const gdn::LaneTable& tl,
                      hipStream_t st) {
  const int rows = p.lanes * (p.draft ? 2 * p.t_max - 1 : p.t_max);
  const long fours = (long)rows * ((p.slices + 3) / 4);
  const bool few = fours < 256;
  const int groups = few ? p.slices : (p.slices + 3) / 4;
  const dim3 grid((unsigned)((long)rows * groups));
  hipError_t e =
      few ? launch(sum_kernel<T, 1>, grid, dim3(kThreads), st, p, tl, groups)
          : launch(sum_kernel<T, 4>, grid, dim3(kThreads), st, p, tl, groups);
  if (e == hipSuccess && p.draft) {
    const int parts = (p.rest_slices + kRestSlices - 1) / kRestSlices;
    e = launch(rest_kernel<T>, dim3((unsigned)((long)p.lanes * parts)),
               dim3(kWide), st, p, tl, parts);
  }
  if (e != hipSuccess) return e;
  return launch(pick_kernel<T>, dim3((unsigned)p.lanes), dim3(kWide), st, p, tl);
}

}  // namespace gdnv

extern "C" size_t gdn_draft_verify_workspace_bytes(int32_t n_lanes,
                                                   int32_t t_max,
                                                   int32_t vocab) {
  using namespace gdnv;
  if (!sizes_ok(n_lanes, t_max, vocab)) return 0;
  return bytes_for(n_lanes, t_max, vocab, slices_for(vocab) + 1);
}

extern "C" int gdn_draft_verify(int32_t n_lanes, int32_t t_max,
                                const int32_t* t_lane, int32_t vocab,
                                const void* logits, int64_t row_stride,
                                const void* draft_logits, int64_t draft_stride,
                                int in_dtype, const int32_t* tokens,
                                const float* uniforms,
                                const float* inv_temperature, int32_t* m_lane,
                                int32_t* next_token, float* accept,
                                void* workspace, size_t ws_bytes,
                                void* stream) {
  using namespace gdnv;
  const int64_t most = (int64_t)1 << 40;
  if (!sizes_ok(n_lanes, t_max, vocab) || row_stride < vocab ||
      row_stride > most || (draft_logits && (draft_stride < vocab || draft_stride > most)))
    return fail(GDN_EINVAL, "gdn_draft_verify: sizes out of range");
  if (in_dtype != GDN_BF16 && in_dtype != GDN_F32)
    return fail(GDN_EINVAL, "gdn_draft_verify: unknown in_dtype");
  if (!t_lane || !logits || !tokens || !uniforms || !inv_temperature ||
      !m_lane || !next_token)
    return fail(GDN_EINVAL, "gdn_draft_verify: required pointer is NULL");
  const int size = in_dtype == GDN_BF16 ? 2 : 4;
  if (misaligned(logits, size) || misaligned(draft_logits, size) ||
      misaligned(tokens, 4) || misaligned(uniforms, 4) ||
      misaligned(inv_temperature, 4) || misaligned(m_lane, 4) ||
      misaligned(next_token, 4) || misaligned(accept, 4) ||
      misaligned(workspace, 16))
    return fail(GDN_EINVAL, "gdn_draft_verify: misaligned pointer");
  const size_t need = gdn_draft_verify_workspace_bytes(n_lanes, t_max, vocab);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_draft_verify: workspace too small");
  gdn::LaneTable tl;
  memset(&tl, 0, sizeof(tl));
  int any = 0;
  for (int n = 0; n < n_lanes; ++n) {
    if (t_lane[n] < 0 || t_lane[n] > t_max)
      return fail(GDN_EINVAL, "gdn_draft_verify: t_lane out of 0..t_max");
    tl.v[n] = (uint8_t)t_lane[n];
    any |= t_lane[n];
  }
  if (!any) return GDN_OK;
  DraftArgs p = {logits, t_max > 1 ? draft_logits : nullptr, tokens, uniforms,
                 inv_temperature, m_lane, next_token, accept, row_stride,
                 draft_stride, n_lanes, t_max, vocab, 0, slices_for(vocab),
                 nullptr, nullptr, nullptr};
  // a row that starts within a line may reach into one slice more
  const auto in_lines = [&](const void* x, int64_t stride) {
    return !misaligned(x, 16) && stride * size % 16 == 0;
  };
  p.slices = slices_for(vocab) +
             (in_lines(logits, row_stride) &&
                      (!p.draft || in_lines(p.draft, draft_stride))
                  ? 0
                  : 1);
  if ((double)n_lanes * (2 * t_max - 1) * p.slices > (double)INT_MAX)
    return fail(GDN_EINVAL, "gdn_draft_verify: grid too large");
  p.parts = (Part*)workspace;
  p.rest = (double*)((char*)workspace +
                     round16((size_t)n_lanes * (2 * t_max - 1) * p.slices * sizeof(Part)));
  p.verdicts = (Verdict*)((char*)p.rest + round16((size_t)n_lanes * p.rest_slices *
                                                  sizeof(double)));
  const hipError_t e = in_dtype == GDN_BF16
                           ? run<uint16_t>(p, tl, (hipStream_t)stream)
                           : run<float>(p, tl, (hipStream_t)stream);
  return gdn::hip_status(e, "gdn_draft_verify launch");
}
