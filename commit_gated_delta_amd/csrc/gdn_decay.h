// gdn_decay.h -- linear attention with a decay per head, in its recurrent
// form (gdn_decay_step) and over packed prompts (gdn_decay_prefill).
// Compiled as part of gdn_prefill.hip.
//
//   S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  a_t = exp(g_t)
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_window_common.h"

namespace gdnd {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Tokens of sequence s are the rows start[s] .. start[s + 1] - 1.
struct SeqTable {
  int start[GDN_MAX_LANES + 1];
};

struct DecayArgs {
  const void *q, *k, *v;
  const float* g;
  const float* s_in;  // NULL: zero states
  float* s_out;       // NULL: not stored
  float* o;           // NULL: not wanted
  float scale;
  int layers, lanes, h_v, h_k, d_v, t_max;
  int per_head;  // g holds one constant per head
};

// ---------------------------------------------------------- recurrent form
// One wave per (head state, 32 columns of d_v): every column of the state is
// independent, so the wave never talks to another one.  Lane (r, c) of 8 x 8
// holds the DK/8 consecutive state rows r at the four columns 4c: 64 f32
// registers at DK = 128, loaded and stored as 128-byte row pieces.  Its k and
// q entries are DK/8 consecutive ones of the token's row.  o needs one sum
// over the eight row groups per token.
constexpr int kStepCols = 32;

template <typename TIn, int R>
__device__ __forceinline__ void load_row(const TIn* __restrict__ p,
                                         float (&x)[R]) {
  if constexpr (sizeof(TIn) == 4) {
    if constexpr (R == 2) {
      const float2 a = *reinterpret_cast<const float2*>(p);
      x[0] = a.x;
      x[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < R / 4; ++i) {
        const f32x4 a = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * i + e] = a[e];
      }
    }
  } else {
    uint32_t w[R / 2];
    if constexpr (R == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (R == 4) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x;
      w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < R / 8; ++i) {
        const u32x4 a = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = a[e];
      }
    }
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Four consecutive columns from column c of a row of n (V4: n % 4 == 0 and
// the row 16-byte (bf16: 8-byte) aligned); columns past the end read as 0.
template <bool V4>
__device__ __forceinline__ f32x4 load_cols(const float* __restrict__ row,
                                           int c, int n) {
  if constexpr (V4) {
    if (c < n) return *reinterpret_cast<const f32x4*>(row + c);
    return f32x4{0.f, 0.f, 0.f, 0.f};
  } else {
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = c + e < n ? row[c + e] : 0.f;
    return x;
  }
}
template <bool V4>
__device__ __forceinline__ f32x4 load_cols(const uint16_t* __restrict__ row,
                                           int c, int n) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if constexpr (V4) {
    if (c < n) {
      const uint2 w = *reinterpret_cast<const uint2*>(row + c);
      x[0] = __uint_as_float(w.x << 16);
      x[1] = __uint_as_float(w.x & 0xffff0000u);
      x[2] = __uint_as_float(w.y << 16);
      x[3] = __uint_as_float(w.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < n) x[e] = __uint_as_float((uint32_t)row[c + e] << 16);
  }
  return x;
}
template <bool V4>
__device__ __forceinline__ void store_cols(float* __restrict__ row, int c,
                                           int n, f32x4 x) {
  if constexpr (V4) {
    if (c < n) *reinterpret_cast<f32x4*>(row + c) = x;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < n) row[c + e] = x[e];
  }
}

// One head's chain over T tokens.  Pointers are at the first token's row of
// the head; qs, vs, gs are the token strides.
template <int DK, typename TIn, bool V4>
__device__ __forceinline__ void decay_chain(
    const TIn* __restrict__ q, const TIn* __restrict__ k,
    const TIn* __restrict__ v, const float* __restrict__ g,
    const float* s_in, float* s_out, float* __restrict__ o, long qs, long vs,
    long gs, int T, int dv, int col0, float scale) {
  constexpr int R = DK / 8;
  const int lane = threadIdx.x & 63;
  const int c = col0 + 4 * (lane & 7), r0 = (lane >> 3) * R;
  f32x4 st[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    st[i] = s_in ? load_cols<V4>(s_in + (long)(r0 + i) * dv, c, dv)
                 : f32x4{0.f, 0.f, 0.f, 0.f};
  for (int t = 0; t < T; ++t) {
    float kk[R], qq[R];
    load_row<TIn, R>(k + t * qs + r0, kk);
    const f32x4 vv = load_cols<V4>(v + t * vs, c, dv);
    const float a = expf(g[t * gs]);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st[i][e] = __builtin_fmaf(kk[i], vv[e], a * st[i][e]);
    if (o) {
      load_row<TIn, R>(q + t * qs + r0, qq);
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(qq[i], st[i][e], y[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[e] += __shfl_xor(y[e], 8);
        y[e] += __shfl_xor(y[e], 16);
        y[e] += __shfl_xor(y[e], 32);
        y[e] *= scale;
      }
      if (lane < 8) store_cols<V4>(o + t * vs, c, dv, y);
    }
  }
  if (s_out) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      store_cols<V4>(s_out + (long)(r0 + i) * dv, c, dv, st[i]);
  }
}

template <int DK, typename TIn, bool V4>
__global__ __launch_bounds__(256) void step_kernel(DecayArgs p,
                                                   gdn::LaneTable tl) {
  const int ncb = (p.d_v + kStepCols - 1) / kStepCols;
  const long unit = (long)blockIdx.x * 4 + threadIdx.x / 64;
  const long item = unit / ncb;
  const int col0 = (int)(unit % ncb) * kStepCols;
  const int h = (int)(item % p.h_v);
  const long lane_of = item / p.h_v;  // layer * lanes + lane
  if (lane_of >= (long)p.layers * p.lanes) return;
  const int n = (int)(lane_of % p.lanes), layer = (int)(lane_of / p.lanes);
  const int T = tl.v[n];
  if (T == 0) return;
  const int hk = h / (p.h_v / p.h_k);
  const long tok = lane_of * p.t_max;
  const long ks = (long)p.h_k * DK, vs = (long)p.h_v * p.d_v;
  const long qo = tok * ks + (long)hk * DK, vo = tok * vs + (long)h * p.d_v;
  const long so = item * DK * p.d_v;
  decay_chain<DK, TIn, V4>(
      (const TIn*)p.q + qo, (const TIn*)p.k + qo, (const TIn*)p.v + vo,
      p.per_head ? p.g + (long)layer * p.h_v + h : p.g + tok * p.h_v + h,
      p.s_in + so, p.s_out ? p.s_out + so : nullptr, p.o ? p.o + vo : nullptr,
      ks, vs, p.per_head ? 0 : p.h_v, T, p.d_v, col0, p.scale);
}

template <int DK, typename TIn, bool V4>
__global__ __launch_bounds__(256) void prompt_chain_kernel(DecayArgs p,
                                                           SeqTable seq) {
  const int ncb = (p.d_v + kStepCols - 1) / kStepCols;
  const long unit = (long)blockIdx.x * 4 + threadIdx.x / 64;
  const long item = unit / ncb;
  const int col0 = (int)(unit % ncb) * kStepCols;
  const int h = (int)(item % p.h_v);
  const long s = item / p.h_v;
  if (s >= p.lanes) return;
  const long tok = seq.start[s];
  const int T = seq.start[s + 1] - seq.start[s];
  const int hk = h / (p.h_v / p.h_k);
  const long ks = (long)p.h_k * DK, vs = (long)p.h_v * p.d_v;
  const long qo = tok * ks + (long)hk * DK, vo = tok * vs + (long)h * p.d_v;
  const long so = item * DK * p.d_v;
  decay_chain<DK, TIn, V4>(
      (const TIn*)p.q + qo, (const TIn*)p.k + qo, (const TIn*)p.v + vo,
      p.per_head ? p.g + h : p.g + tok * p.h_v + h,
      p.s_in ? p.s_in + so : nullptr, p.s_out ? p.s_out + so : nullptr,
      p.o ? p.o + vo : nullptr, ks, vs, p.per_head ? 0 : p.h_v, T, p.d_v, col0,
      p.scale);
}

// ---------------------------------------------------------------- host side
static int check_heads(const char* fn, int h_v, int h_k, int d_k, int d_v) {
  char msg[128];
  if (h_v < 1 || h_k < 1 || h_v % h_k != 0 || d_k < 1 || d_v < 1 ||
      d_v > 1024) {
    snprintf(msg, sizeof(msg), "%s: sizes out of range", fn);
    return fail(GDN_EINVAL, msg);
  }
  if (d_k != 16 && d_k != 32 && d_k != 64 && d_k != 128) {
    snprintf(msg, sizeof(msg), "%s: d_k must be 16, 32, 64 or 128", fn);
    return fail(GDN_EUNSUPPORTED, msg);
  }
  return GDN_OK;
}

static int check_pointers(const char* fn, const DecayArgs& p, int in_dtype) {
  char msg[128];
  const char* what = nullptr;
  if (!p.k || !p.v || !p.g || (p.o && !p.q)) what = "required pointer is NULL";
  else if (in_dtype != GDN_BF16 && in_dtype != GDN_F32) what = "unknown in_dtype";
  else if (misaligned(p.q, 16) || misaligned(p.k, 16) || misaligned(p.v, 16) ||
           misaligned(p.g, 16) || misaligned(p.s_in, 16) ||
           misaligned(p.s_out, 16) || misaligned(p.o, 16))
    what = "pointers must be 16-byte aligned";
  if (!what) return GDN_OK;
  snprintf(msg, sizeof(msg), "%s: %s", fn, what);
  return fail(GDN_EINVAL, msg);
}

// Calls f with the element type, d_k and column access of a call as types.
template <typename F>
static hipError_t by_shape(int d_k, int d_v, int in_dtype, F&& f) {
  auto of_type = [&](auto dk, auto t) {
    if (d_v % 4 == 0) return f(dk, t, std::true_type{});
    return f(dk, t, std::false_type{});
  };
  auto of_dk = [&](auto dk) {
    if (in_dtype == GDN_BF16) return of_type(dk, uint16_t{});
    return of_type(dk, float{});
  };
  switch (d_k) {
    case 16: return of_dk(std::integral_constant<int, 16>{});
    case 32: return of_dk(std::integral_constant<int, 32>{});
    case 64: return of_dk(std::integral_constant<int, 64>{});
    default: return of_dk(std::integral_constant<int, 128>{});
  }
}

// Workgroups of four waves for one wave per (state, 32 columns).
static long step_blocks(long states, int d_v) {
  const long units = states * ((d_v + kStepCols - 1) / kStepCols);
  return (units + 3) / 4;
}

// Prefix sums of the sequence lengths; the number of tokens, or -1.
static long seq_starts(int32_t n_seqs, const int32_t* seq_len, SeqTable& t) {
  if (n_seqs < 1 || n_seqs > GDN_MAX_LANES || !seq_len) return -1;
  memset(&t, 0, sizeof(t));
  long sum = 0;
  for (int i = 0; i < n_seqs; ++i) {
    if (seq_len[i] < 0) return -1;
    sum += seq_len[i];
    if (sum > INT_MAX) return -1;
    t.start[i + 1] = (int)sum;
  }
  return sum;
}

}  // namespace gdnd

extern "C" int gdn_decay_step(const gdn_dims* dims, const int32_t* t_lane,
                              const void* q, const void* k, const void* v,
                              int in_dtype, const float* g, float* S, float* o,
                              float scale, int flags, void* stream) {
  using namespace gdnd;
  const char* fn = "gdn_decay_step";
  int rc = gdn::check_dims(dims);
  if (rc != GDN_OK) return rc;
  const gdn_dims& d = *dims;
  if (flags & ~(GDN_FLAG_HEAD_DECAY | GDN_FLAG_KEEP_STATE))
    return fail(GDN_EINVAL, "gdn_decay_step: unknown flag bits");
  const bool keep = flags & GDN_FLAG_KEEP_STATE;
  if (!t_lane || !S)
    return fail(GDN_EINVAL, "gdn_decay_step: required pointer is NULL");
  if (keep && !o)
    return fail(GDN_EINVAL,
                "gdn_decay_step: neither the state nor outputs are wanted");
  DecayArgs p = {q, k, v, g, S, keep ? nullptr : S, o, scale, d.n_layers,
                 d.n_lanes, d.h_v, d.h_k, d.d_v, d.t_max,
                 (flags & GDN_FLAG_HEAD_DECAY) ? 1 : 0};
  rc = check_pointers(fn, p, in_dtype);
  if (rc != GDN_OK) return rc;
  gdn::LaneTable tl;
  memset(&tl, 0, sizeof(tl));
  int any = 0;
  for (int n = 0; n < d.n_lanes; ++n) {
    if (t_lane[n] < 0 || t_lane[n] > d.t_max)
      return fail(GDN_EINVAL, "gdn_decay_step: t_lane out of 0..t_max");
    tl.v[n] = (uint8_t)t_lane[n];
    any |= t_lane[n];
  }
  if (!any) return GDN_OK;
  const long blocks =
      step_blocks((long)d.n_layers * d.n_lanes * d.h_v, d.d_v);
  if (blocks > INT_MAX)
    return fail(GDN_EINVAL, "gdn_decay_step: grid too large");
  const hipError_t e = by_shape(
      d.d_k, d.d_v, in_dtype, [&](auto dk, auto t, auto v4) {
        return launch(step_kernel<decltype(dk)::value, decltype(t),
                                  decltype(v4)::value>,
                      dim3((unsigned)blocks), dim3(256), (hipStream_t)stream,
                      p, tl);
      });
  return gdn::hip_status(e, "gdn_decay_step launch");
}

extern "C" size_t gdn_decay_prefill_workspace_bytes(int32_t n_seqs,
                                                    const int32_t* seq_len,
                                                    int32_t h_v, int32_t h_k,
                                                    int32_t d_k, int32_t d_v) {
  using namespace gdnd;
  SeqTable t;
  if (check_heads("gdn_decay_prefill_workspace_bytes", h_v, h_k, d_k, d_v) !=
          GDN_OK ||
      seq_starts(n_seqs, seq_len, t) < 0)
    return 0;
  return 0;
}

extern "C" int gdn_decay_prefill(int32_t n_seqs, const int32_t* seq_len,
                                 int32_t h_v, int32_t h_k, int32_t d_k,
                                 int32_t d_v, const void* q, const void* k,
                                 const void* v, int in_dtype, const float* g,
                                 const float* S_init, float* S_final, float* o,
                                 void* workspace, size_t ws_bytes, float scale,
                                 int flags, void* stream) {
  using namespace gdnd;
  const char* fn = "gdn_decay_prefill";
  int rc = check_heads(fn, h_v, h_k, d_k, d_v);
  if (rc != GDN_OK) return rc;
  SeqTable seq;
  const long tokens = seq_starts(n_seqs, seq_len, seq);
  if (tokens < 0)
    return fail(GDN_EINVAL, "gdn_decay_prefill: bad n_seqs or seq_len");
  if (flags & ~GDN_FLAG_HEAD_DECAY)
    return fail(GDN_EINVAL, "gdn_decay_prefill: unknown flag bits");
  if (!o && !S_final)
    return fail(GDN_EINVAL,
                "gdn_decay_prefill: neither states nor outputs are wanted");
  DecayArgs p = {q, k, v, g, S_init, S_final, o, scale, 1, n_seqs, h_v, h_k,
                 d_v, 0, (flags & GDN_FLAG_HEAD_DECAY) ? 1 : 0};
  rc = check_pointers(fn, p, in_dtype);
  if (rc != GDN_OK) return rc;
  const size_t need =
      gdn_decay_prefill_workspace_bytes(n_seqs, seq_len, h_v, h_k, d_k, d_v);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_decay_prefill: workspace too small");
  if (need > 0 && misaligned(workspace, 16))
    return fail(GDN_EINVAL,
                "gdn_decay_prefill: pointers must be 16-byte aligned");
  if (tokens == 0 && !S_final) return GDN_OK;
  const double units = (double)n_seqs * h_v * ((d_v + kStepCols - 1) / kStepCols);
  if (units > (double)INT_MAX)
    return fail(GDN_EINVAL, "gdn_decay_prefill: grid too large");
  const long blocks = step_blocks((long)n_seqs * h_v, d_v);
  const hipError_t e =
      by_shape(d_k, d_v, in_dtype, [&](auto dk, auto t, auto v4) {
        return launch(prompt_chain_kernel<decltype(dk)::value, decltype(t),
                                          decltype(v4)::value>,
                      dim3((unsigned)blocks), dim3(256), (hipStream_t)stream,
                      p, seq);
      });
  return gdn::hip_status(e, "gdn_decay_prefill launch");
}
