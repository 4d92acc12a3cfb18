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
// Which drafts stand needs every row but the last, so their sums are f32 at
// the memory's rate (a chance is 2 steps of 2^-24 off, rms, and 1e-8 in f64).  The next token is where a running sum passes a given
// number, and an error d of the sums moves it with a chance of about d times
// the number of likely tokens: the one row that it is sampled from is summed
// up again in f64.
#pragma once
#include <hip/hip_runtime.h>

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
// one) and the sum of 2^((x - m) c) with that as m.
struct Part {
  float m, z;
};
// The same of a slice of the row that the next token is sampled from, without
// the id that it cannot be.
struct Exact {
  double z;
  float m;
  int pad;
};

// What a lane's drafts come to.
struct Verdict {
  int m;   // accepted prefix, the anchor included
  int ok;  // the rows that a draft fell at have distributions
};

// Of the rows that a fallen draft and its drafter's distribution leave: the
// largest logits and the reciprocals of the sums.
struct Left {
  double top, draft_top, f, draft_f;
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
  int groups;      // slices of a row in `parts`, of kGroup ids
  int slices;      // slices of a row in `exact`, of kSlice ids; both count from
                   // the 16-byte line that a row starts in
  Part* parts;     // [target rows 0 .. t_max - 2, then drafter's rows][groups]
  Exact* exact;    // [lanes][target's row, drafter's][slices]
  double* rest;    // [lanes][slices]: sums of max(p - q, 0), from the first id on
  Verdict* verdicts;  // [lanes]
  Left* left;         // [lanes]
};

constexpr int kSlice = 2048, kGroup = 8192;
constexpr int kThreads = 256;  // of sum_kernel and rest_kernel
constexpr int kExact = 512;    // of exact_kernel
constexpr int kPick = 1024;    // of pick_kernel

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

// A workgroup's share of a row: N logits a thread from line `first_line` on
// (threads take vectors in turn), masked past the row's ends.
template <typename T, int N, int THREADS>
struct Share {
  static constexpr int E = 16 / sizeof(T), V = N / E;
  float x[V][E];
  int first, skew;  // this thread's first line

  __device__ __forceinline__ void load(const T* row, int vocab, int first_line) {
    skew = skew_of(row);
    first = first_line + threadIdx.x;
    const u32x4* line = reinterpret_cast<const u32x4*>(row - skew);
    const int lines = (vocab + skew + E - 1) / E;
    u32x4 raw[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = first + k * THREADS;
      raw[k] = line[i < lines ? i : lines - 1];
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int i = first + k * THREADS;
      const int id = i < lines ? i * E - skew : vocab;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (sizeof(T) == 4) x[k][e] = __uint_as_float(raw[k][e]);
        else
          x[k][e] = __uint_as_float(e & 1 ? raw[k][e / 2] & 0xffff0000u
                                          : raw[k][e / 2] << 16);
      }
      if (id < 0 || id > vocab - E) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((unsigned)(id + e) >= (unsigned)vocab) x[k][e] = -INFINITY;
      }
    }
  }
  __device__ __forceinline__ float most() const {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) m = nan_max(m, x[k][e]);
    return m;
  }
  __device__ __forceinline__ void leave_out(int id) {
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((first + k * THREADS) * E - skew + e == id) x[k][e] = -INFINITY;
  }
};

// Sums of the rows that decide about the drafts: a workgroup per kGroup ids,
// read once into registers, so that its largest logit is known before its sum
// and no exponential is taken twice.  Bound by HBM: 8 lanes of up to 15 drafts,
// 131072 ids in f32, drafter's rows too: 10.5 us, 45 MB at 4.3 TB/s; 64 lanes
// of up to 5, bf16: 11.5 us, 46 MB at 4.0, the vector units nearly full.
// (In f64 18 and 32 us, 26 vector instructions a logit.)
template <typename T>
__global__ __launch_bounds__(kThreads, 4) void sum_kernel(DraftArgs p,
                                                          gdn::LaneTable tl) {
  constexpr int N = kGroup / kThreads;
  __shared__ float tops[4], sums[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = blockIdx.x / p.groups, part = blockIdx.x % p.groups;
  const int per = p.t_max - 1, targets = p.lanes * per;
  const bool drafter = row >= targets;
  const int n = (drafter ? row - targets : row) / per;
  const int t = (drafter ? row - targets : row) % per;
  if (t >= tl.v[n] - 1) return;
  Share<T, N, kThreads> s;
  s.load(drafter ? drafter_row<T>(p, n, t) : target_row<T>(p, n, t), p.vocab,
         part * (kGroup / Share<T, N, kThreads>::E));
  const double c = exponent_of(p, n);
  float m = wave_nan_max(s.most());
  if (lane == 0) tops[wave] = m;
  __syncthreads();
  m = nan_max(nan_max(tops[0], tops[1]), nan_max(tops[2], tops[3]));
  // c in two parts: rounded to one it would tilt the exponents of far logits.
  // Both are positive, so that a logit of -inf stays one.
  const float ref = m == -INFINITY ? 0.f : m;
  float hi = (float)c;
  if ((double)hi > c) hi = __uint_as_float(__float_as_uint(hi) - 1);
  const float lo = fmaxf((float)(c - (double)hi), 1.17549435e-38f);
  float z = 0.f;
#pragma unroll
  for (int k = 0; k < s.V; ++k)
#pragma unroll
    for (int e = 0; e < s.E; ++e) {
      const float d = s.x[k][e] - ref;
      z += __builtin_amdgcn_exp2f(__builtin_fmaf(d, hi, d * lo));
    }
  z = gdn::wave_sum(z);
  if (lane == 0) sums[wave] = z;
  __syncthreads();
  if (tid == 0)
    p.parts[(long)row * p.groups + part] = {
        m, (sums[0] + sums[1]) + (sums[2] + sums[3])};
}

// Slices of kGroup ids a row from which the verdicts and both rows' sums are
// worked out once a lane, by launches of their own (2^20 ids).  Below, every
// workgroup that needs them works them out for itself: that saves launches, but
// its work grows with the square of the vocabulary.  With and without launches
// of their own, drafter's rows given, bf16: one lane of one draft over 2^19,
// 2^20, 2^21 ids 22, 27, 42 and 19, 24, 58 us; 8 lanes of 15 73, 136, 256 and 83,
// 182, 440; 64 lanes of 5 225, 444, 867 and 308, 741, 1923.
constexpr int kManyGroups = 128;

// A workgroup of kExact threads works a lane's verdict out from the slices'
// sums, a wave a row.
struct Rows {
  float m[2][GDN_MAX_T];
  double z[2][GDN_MAX_T];
  Verdict verdict;
};
template <typename T>
__device__ __forceinline__ Verdict decide(const DraftArgs& p, int n, int T_n,
                                          double c, Rows& rows, bool write) {
  const int lane = threadIdx.x & 63, wave = gdn::uniform(threadIdx.x >> 6);
  const int drafts = T_n - 1;
  // the first wave's lanes hold a draft each: its logits are on their way
  // while the rows are summed up
  const bool drafted = wave == 0 && lane < drafts;
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
  const int count = p.draft ? 2 * drafts : drafts;
  auto parts_of = [&](int r) {
    const int d = r >= drafts ? 1 : 0;
    return p.parts + (((long)d * p.lanes + n) * (p.t_max - 1) + r - d * drafts) * p.groups;
  };
  constexpr int kStep = kExact / 64;
  const Part none = {-INFINITY, 0.f};
  Part next = none;
  if (wave < count && lane < p.groups) next = parts_of(wave)[lane];
  for (int r = wave; r < count; r += kStep) {
    const Part* parts = parts_of(r);
    const Part first = next;
    next = none;
    if (r + kStep < count && lane < p.groups) next = parts_of(r + kStep)[lane];
    float m = first.m;
    for (int i = lane + 64; i < p.groups; i += 64) m = nan_max(m, parts[i].m);
    m = wave_nan_max(m);
    const double ref = m == -INFINITY ? 0.0 : (double)m;
    double z = first.z * weight_of(first.m, ref, c);
    for (int i = lane + 64; i < p.groups; i += 64)
      z += parts[i].z * weight_of(parts[i].m, ref, c);
    z = wave_sum64(z);
    if (lane == 0) {
      const int d = r >= drafts;
      rows.m[d][r - d * drafts] = m;
      rows.z[d][r - d * drafts] = z;
    }
  }
  __syncthreads();
  if (wave == 0) {
    bool stands = true, ok = true;  // (lanes past the drafts)
    if (drafted) {
      const float m = rows.m[0][lane];
      ok = c > 0.0 && fabsf(m) < INFINITY;
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
    const uint64_t fell = __ballot(!stands), good = __ballot(ok);
    if (lane == 0) {
      const int first = fell ? __builtin_ctzll(fell) : drafts;
      rows.verdict = {first + 1, (int)(good >> first & 1)};
    }
  }
  __syncthreads();
  return rows.verdict;
}

// The verdicts alone, a workgroup per lane.
template <typename T>
__global__ __launch_bounds__(kExact) void verdict_kernel(DraftArgs p,
                                                         gdn::LaneTable tl) {
  __shared__ Rows rows;
  const int n = blockIdx.x, T_n = tl.v[n];
  if (T_n == 0) return;
  Verdict v = {1, 1};
  if (T_n > 1) v = decide<T>(p, n, T_n, exponent_of(p, n), rows, true);
  if (threadIdx.x == 0) p.verdicts[n] = v;
}

// f64 sums by slices of the row that the next token is sampled from (leaving
// the fallen draft out, where it has no distribution), or of the drafter's row
// beside it, and unless they are KNOWN the verdicts.  A workgroup takes kGroup
// ids.  Bound by the verdicts' chain of loads and, with many lanes, by the
// exponentials in f64: 8 lanes and their drafter's rows 8.1 us, 64 lanes 13.4.
template <typename T, bool KNOWN>
__global__ __launch_bounds__(kExact) void exact_kernel(DraftArgs p,
                                                      gdn::LaneTable tl,
                                                      int sides) {
  constexpr int N = kGroup / kExact, kSlices = kGroup / kSlice;
  typedef Share<T, N, kExact> S;
  constexpr int kVectors = kSlice / S::E;  // of a slice
  __shared__ Rows rows;
  __shared__ float tops[kExact / 64];
  __shared__ double sums[kSlices][kVectors];
  const int part = blockIdx.x % p.groups;
  const int side = blockIdx.x / p.groups % sides;
  const int n = blockIdx.x / p.groups / sides, T_n = tl.v[n];
  if (T_n == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  const double c = exponent_of(p, n);
  Verdict v = {1, 1};
  if constexpr (KNOWN) {
    v = p.verdicts[n];
  } else {
    if (T_n > 1) v = decide<T>(p, n, T_n, c, rows, part == 0 && side == 0);
    if (part == 0 && side == 0 && tid == 0) p.verdicts[n] = v;
  }
  const bool fell = v.m < T_n;
  if (!v.ok || (side == 1 && !fell)) return;
  S s;
  s.load(side ? drafter_row<T>(p, n, v.m - 1) : target_row<T>(p, n, v.m - 1),
         p.vocab, part * (kGroup / S::E));
  float m = wave_nan_max(s.most());
  if (lane == 0) tops[wave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kExact / 64; ++i) m = nan_max(m, tops[i]);
  const double ref = m == -INFINITY ? 0.0 : (double)m;
  if (fell && !p.draft) s.leave_out(p.tokens[(long)n * p.t_max + v.m]);
#pragma unroll
  for (int k = 0; k < S::V; ++k) {
    double z[2] = {0.0, 0.0};
#pragma unroll
    for (int e = 0; e < S::E; ++e)
      z[e & 1] += weight_in_sum(s.x[k][e], ref, c);
    const int at = k * kExact + tid;  // of the group's vectors
    sums[at / kVectors][at % kVectors] = z[0] + z[1];
  }
  __syncthreads();
  const int slice = part * kSlices + wave;  // a wave adds one up
  if (wave >= kSlices || slice >= p.slices) return;
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < kVectors / 64; ++i) z += sums[wave][64 * i + lane];
  z = or_nothing(wave_sum64(z));
  if (lane == 0)
    p.exact[((long)n * 2 + side) * p.slices + slice] = {z, m, 0};
}

// A row of `exact`: its largest logit and the sum of its weights to that.
// Every wave works it out for itself.
__device__ __forceinline__ void whole_row(const Exact* e, int slices, double c,
                                          float& m, double& z) {
  const int lane = threadIdx.x & 63;
  m = -INFINITY;
  for (int i = lane; i < slices; i += 64) m = nan_max(m, e[i].m);
  m = wave_nan_max(m);
  const double ref = m == -INFINITY ? 0.0 : (double)m;
  z = 0.0;
  for (int i = lane; i < slices; i += 64) z += e[i].z * weight_of(e[i].m, ref, c);
  z = wave_sum64(z);
}

// max(p - q, 0) of an id.
__device__ __forceinline__ double weight_left(const Left& r, float x, float y,
                                              double c) {
  const double w = weight_of(x, r.top, c) * r.f -
                   weight_of(y, r.draft_top, c) * r.draft_f;
  return w > 0.0 ? w : 0.0;
}

// Both rows' largest logits and sums alone, a workgroup per lane: one half of
// it for the target's row, the other for the drafter's.
template <typename T>
__global__ __launch_bounds__(kPick) void left_kernel(DraftArgs p,
                                                     gdn::LaneTable tl) {
  constexpr int kHalf = kPick / 2, kWaves = kHalf / 64;
  __shared__ float tops[2][kWaves];
  __shared__ double sums[2][kWaves];
  const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int side = gdn::uniform(tid / kHalf), wave = gdn::uniform(tid % kHalf >> 6);
  if (tl.v[n] < 2) return;
  const Verdict v = p.verdicts[n];
  if (!v.ok || v.m == tl.v[n]) return;
  const double c = exponent_of(p, n);
  const Exact* e = p.exact + ((long)n * 2 + side) * p.slices;
  float m = -INFINITY;
  for (int i = tid % kHalf; i < p.slices; i += kHalf) m = nan_max(m, e[i].m);
  m = wave_nan_max(m);
  if (lane == 0) tops[side][wave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i) m = nan_max(m, tops[side][i]);
  const double ref = m == -INFINITY ? 0.0 : (double)m;
  double z = 0.0;
  for (int i = tid % kHalf; i < p.slices; i += kHalf)
    z += e[i].z * weight_of(e[i].m, ref, c);
  z = wave_sum64(z);
  if (lane == 0) sums[side][wave] = z;
  __syncthreads();
  if (tid % kHalf != 0) return;
  z = 0.0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) z += sums[side][i];
  Left& r = p.left[n];
  if (side == 0) {
    r.top = m;
    r.f = 1.0 / z;
  } else {
    r.draft_top = m;
    r.draft_f = 1.0 / z;
  }
}

// With a drafter's distribution: sums of max(p - q, 0) by slices of the row
// where a draft fell.  The logits, in the cache still, are on their way while
// the sums of both rows are worked out, unless these are KNOWN.  8 lanes: 5.6
// us, bound by latency.
template <typename T, bool KNOWN>
__global__ __launch_bounds__(kThreads) void rest_kernel(DraftArgs p,
                                                        gdn::LaneTable tl) {
  constexpr int N = kSlice / kThreads;
  __shared__ double sums[kThreads / 64];
  const int n = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const int tid = threadIdx.x;
  if (tl.v[n] < 2) return;
  const Verdict v = p.verdicts[n];
  if (!v.ok || v.m == tl.v[n]) return;
  const T* row = target_row<T>(p, n, v.m - 1);
  const T* drafter = drafter_row<T>(p, n, v.m - 1);
  float x[N], y[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = slice * kSlice + k * kThreads + tid;
    x[k] = y[k] = -INFINITY;
    if (i < p.vocab) {
      x[k] = logit_at(row, i);
      y[k] = logit_at(drafter, i);
    }
  }
  const double c = exponent_of(p, n);
  Left r;
  if constexpr (KNOWN) {
    r = p.left[n];
  } else {
    const Exact* e = p.exact + (long)n * 2 * p.slices;
    float m, dm;
    double z, dz;
    whole_row(e, p.slices, c, m, z);
    whole_row(e + p.slices, p.slices, c, dm, dz);
    r = {m, dm, 1.0 / z, 1.0 / dz};
    if (slice == 0 && tid == 0) p.left[n] = r;
  }
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < N; ++k) sum += weight_left(r, x[k], y[k], c);
  sum = wave_sum64(sum);
  if (tid % 64 == 0) sums[tid / 64] = sum;
  __syncthreads();
  if (tid == 0)
    p.rest[(long)n * p.slices + slice] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// The next token, a workgroup per lane: the slice that the border lies in,
// then the id within it.
// 5.6 to 6.6 us for 1 to 64 lanes, bound by latency: three passes over the
// slices' sums, one over a slice.
template <typename T>
__global__ __launch_bounds__(kPick) void pick_kernel(DraftArgs p,
                                                     gdn::LaneTable tl) {
  __shared__ double sums[kPick / 64];
  __shared__ double found[2];  // the running sum before the slice, and the border
  __shared__ int which, first_id[kPick / 64], last_id[kPick / 64];
  const int n = blockIdx.x, T_n = tl.v[n];
  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  if (T_n == 0) return;
  const double c = exponent_of(p, n);
  const Verdict v = p.verdicts[n];
  const bool fell = v.m < T_n;
  const Exact* e = p.exact + (long)n * 2 * p.slices;
  Left r;
  float top = NAN;
  if (v.ok && fell && p.draft) {
    r = p.left[n];
    top = (float)r.top;
  } else if (v.ok) {
    double z;
    whole_row(e, p.slices, c, top, z);
  }
  if (!v.ok || !(c > 0.0) || !(fabsf(top) < INFINITY)) {
    if (tid == 0) {
      p.m[n] = v.m;
      p.next[n] = -1;
    }
    return;
  }
  if (wave == 0) {
    bool rest = fell && p.draft;
    const float u = p.uniforms[(long)n * p.t_max + T_n - 1];
    const double share = u > 0.f ? u < 1.f ? (double)u : 1.0 : 0.0;
    auto slice_sum = [&](int i) {
      if (i >= p.slices) return 0.0;
      if (rest) return p.rest[(long)n * p.slices + i];
      return or_nothing(e[i].z * weight_of(e[i].m, top, c));
    };
    for (;;) {
      double whole = 0.0;
      for (int i0 = 0; i0 < p.slices; i0 += 64)
        whole += lane_value(wave_scan64(slice_sum(i0 + lane)), 63);
      if (whole == 0.0 && rest) {  // nothing is left: from p
        rest = false;
        continue;
      }
      const double border = share * whole;
      double before = 0.0, base = 0.0, last_base = 0.0;
      int got = -1, last = -1;
      for (int i0 = 0; i0 < p.slices && got < 0; i0 += 64) {
        const double x = slice_sum(i0 + lane);
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
        which = (got >= 0 ? got : last) * 2 + (rest ? 1 : 0);
        found[0] = got >= 0 ? base : last_base;
        found[1] = border;
      }
      break;
    }
  }
  __syncthreads();
  if (which < 0) {  // p is nothing but the draft that fell to rounding
    if (tid == 0) {
      p.m[n] = v.m;
      p.next[n] = p.tokens[(long)n * p.t_max + v.m];
    }
    return;
  }
  const bool rest = which & 1;
  const T* row = target_row<T>(p, n, v.m - 1);
  const int gone = fell && !p.draft ? p.tokens[(long)n * p.t_max + v.m] : -1;
  // ids of the slice, consecutive ones a thread
  constexpr int kPer = kSlice / kPick;
  const int from = (which >> 1) * kSlice - (rest ? 0 : skew_of(row)) + tid * kPer;
  double mine = 0.0;
  double x[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = from + k;
    x[k] = 0.0;
    if ((unsigned)i < (unsigned)p.vocab && i != gone)
      x[k] = rest ? weight_left(r, logit_at(row, i),
                                logit_at(drafter_row<T>(p, n, v.m - 1), i), c)
                  : weight_of(logit_at(row, i), top, c);
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
  for (int i = 0; i < kPick / 64 && token < 0; ++i) token = first_id[i];
  for (int i = kPick / 64 - 1; i >= 0 && token < 0; --i) token = last_id[i];
  p.m[n] = v.m;
  p.next[n] = token;
}

// ---------------------------------------------------------------- host side
static bool sizes_ok(int32_t n_lanes, int32_t t_max, int32_t vocab) {
  return n_lanes >= 1 && n_lanes <= GDN_MAX_LANES && t_max >= 1 &&
         t_max <= GDN_MAX_T && vocab >= 1 && vocab <= 1 << 30;
}
static int slices_for(int32_t vocab, int ids) { return (vocab + ids - 1) / ids; }
// Offsets of the workspace's parts, with `more` slices a row than its ids fill
// (a row that starts within a line may reach into one more).
struct Layout {
  int groups, slices;
  size_t exact, rest, verdicts, left, all;
};
static Layout layout_of(int32_t n_lanes, int32_t t_max, int32_t vocab,
                        int more) {
  Layout l;
  l.groups = slices_for(vocab, kGroup) + more;
  l.slices = slices_for(vocab, kSlice) + more;
  l.exact = round16((size_t)n_lanes * 2 * (t_max - 1) * l.groups * sizeof(Part));
  l.rest = l.exact + round16((size_t)n_lanes * 2 * l.slices * sizeof(Exact));
  l.verdicts = l.rest + round16((size_t)n_lanes * l.slices * sizeof(double));
  l.left = l.verdicts + round16((size_t)n_lanes * sizeof(Verdict));
  l.all = l.left + round16((size_t)n_lanes * sizeof(Left));
  return l;
}

template <typename T>
static hipError_t run(const DraftArgs& p, const gdn::LaneTable& tl,
                      hipStream_t st) {
  const int sides = p.draft ? 2 : 1;
  hipError_t e = hipSuccess;
  if (p.t_max > 1)
    e = launch(sum_kernel<T>,
               dim3((unsigned)((long)p.lanes * (p.t_max - 1) * sides * p.groups)),
               dim3(kThreads), st, p, tl);
  const bool known = p.t_max > 1 && p.groups >= kManyGroups;
  if (e == hipSuccess && known)
    e = launch(verdict_kernel<T>, dim3((unsigned)p.lanes), dim3(kExact), st, p, tl);
  const dim3 exact((unsigned)((long)p.lanes * sides * p.groups));
  if (e == hipSuccess)
    e = known ? launch(exact_kernel<T, true>, exact, dim3(kExact), st, p, tl, sides)
              : launch(exact_kernel<T, false>, exact, dim3(kExact), st, p, tl, sides);
  if (e == hipSuccess && p.draft) {
    const dim3 rest((unsigned)((long)p.lanes * p.slices));
    if (known) {
      e = launch(left_kernel<T>, dim3((unsigned)p.lanes), dim3(kPick), st, p, tl);
      if (e == hipSuccess)
        e = launch(rest_kernel<T, true>, rest, dim3(kThreads), st, p, tl);
    } else {
      e = launch(rest_kernel<T, false>, rest, dim3(kThreads), st, p, tl);
    }
  }
  if (e != hipSuccess) return e;
  return launch(pick_kernel<T>, dim3((unsigned)p.lanes), dim3(kPick), st, p, tl);
}

}  // namespace gdnv

extern "C" size_t gdn_draft_verify_workspace_bytes(int32_t n_lanes,
                                                   int32_t t_max,
                                                   int32_t vocab) {
  using namespace gdnv;
  if (!sizes_ok(n_lanes, t_max, vocab)) return 0;
  return layout_of(n_lanes, t_max, vocab, 1).all;
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
                 draft_stride, n_lanes, t_max, vocab, 0, 0, nullptr, nullptr,
                 nullptr, nullptr, nullptr};
  const auto in_lines = [&](const void* x, int64_t stride) {
    return !misaligned(x, 16) && stride * size % 16 == 0;
  };
  const Layout l = layout_of(
      n_lanes, t_max, vocab,
      in_lines(logits, row_stride) &&
              (!p.draft || in_lines(p.draft, draft_stride))
          ? 0
          : 1);
  // threads of the largest launch (of sum_kernel, exact_kernel, rest_kernel)
  const double groups = (double)n_lanes * (p.draft ? 2 : 1) * l.groups;
  const double threads = fmax(fmax(groups * (t_max - 1) * kThreads, groups * kExact),
                              (double)n_lanes * l.slices * kThreads);
  if (threads > (double)UINT32_MAX ||
      (double)n_lanes * 2 * t_max * l.slices > (double)INT_MAX)
    return fail(GDN_EINVAL, "gdn_draft_verify: grid too large");
  p.groups = l.groups;
  p.slices = l.slices;
  p.parts = (Part*)workspace;
  p.exact = (Exact*)((char*)workspace + l.exact);
  p.rest = (double*)((char*)workspace + l.rest);
  p.verdicts = (Verdict*)((char*)workspace + l.verdicts);
  p.left = (Left*)((char*)workspace + l.left);
  const hipError_t e = in_dtype == GDN_BF16
                           ? run<uint16_t>(p, tl, (hipStream_t)stream)
                           : run<float>(p, tl, (hipStream_t)stream);
  return gdn::hip_status(e, "gdn_draft_verify launch");
}
