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
};

constexpr int kBlock = 1024;

__device__ __forceinline__ double block_sum(double x, double* red) {
  for (int i = 32; i > 0; i /= 2) x += __shfl_xor(x, i);
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = x;
  __syncthreads();
  double s = 0;
  for (int i = 0; i < kBlock / 64; ++i) s += red[i];
  return s;
}
// The largest logit of a row (NaN if it holds one).
template <typename T>
__device__ __forceinline__ float row_max(const T* x, int vocab, float* red) {
  float m = -INFINITY;
  for (int i = threadIdx.x; i < vocab; i += kBlock)
    m = __builtin_elementwise_maximum(m, logit_at(x, i));
  for (int i = 32; i > 0; i /= 2) m = __builtin_elementwise_maximum(m, __shfl_xor(m, i));
  __syncthreads();
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = m;
  __syncthreads();
  m = red[0];
  for (int i = 1; i < kBlock / 64; ++i) m = __builtin_elementwise_maximum(m, red[i]);
  return m;
}

// One workgroup per lane, every sum in f64.
template <typename T>
__global__ __launch_bounds__(kBlock) void verify_kernel(DraftArgs p,
                                                        gdn::LaneTable tl) {
  __shared__ double red[kBlock];
  const int n = blockIdx.x, tid = threadIdx.x, V = p.vocab, T_n = tl.v[n];
  if (T_n == 0) return;
  const double it = p.it[n];
  const bool it_ok = p.it[n] >= 1e-30f && p.it[n] <= 1e30f;
  auto target = [&](int t) { return (const T*)p.logits + ((long)n * p.t_max + t) * p.stride; };
  auto drafter = [&](int t) { return (const T*)p.draft + ((long)n * (p.t_max - 1) + t) * p.draft_stride; };
  auto chance = [&](const T* x, long i, double m) { return exp(((double)logit_at(x, i) - m) * it); };
  // the row's largest logit and the sum of its exponentials; false: it has
  // no distribution
  auto sums = [&](const T* x, double& m, double& z) {
    m = row_max(x, V, (float*)red);
    if (!it_ok || !(fabs(m) < INFINITY)) return false;
    double s = 0;
    for (int i = tid; i < V; i += kBlock) s += chance(x, i, m);
    z = block_sum(s, red);
    return true;
  };
  int m = 1;
  bool open = true;
  double zm, z, dm = 0, dz = 1;
  for (int t = 0; t < T_n - 1; ++t) {
    bool ok = sums(target(t), zm, z);
    if (p.draft) ok &= sums(drafter(t), dm, dz);
    const int w = p.tokens[(long)n * p.t_max + t + 1];
    double pw = 0, qw = 1;
    if ((unsigned)w < (unsigned)V && ok) {
      pw = chance(target(t), w, zm) / z;
      if (p.draft) qw = chance(drafter(t), w, dm) / dz;
    }
    if (open && ok && (double)p.uniforms[(long)n * p.t_max + t] * qw < pw) ++m;
    else open = false;
    if (p.accept && tid == 0)
      p.accept[(long)n * p.t_max + t] = !ok ? NAN : pw == 0 ? 0.f : pw >= qw ? 1.f : (float)(pw / qw);
  }
  const int t = m - 1;
  bool ok = sums(target(t), zm, z);
  const bool fell = m < T_n;
  if (fell && p.draft) ok &= sums(drafter(t), dm, dz);
  const int w = fell ? p.tokens[(long)n * p.t_max + t + 1] : -1;
  if (!ok) {
    if (tid == 0) {
      p.m[n] = m;
      p.next[n] = -1;
    }
    return;
  }
  bool rest = fell;
  auto weight = [&](int i) {
    double x = chance(target(t), i, zm) / z;
    if (rest) {
      if (!p.draft) x = i == w ? 0 : x;
      else x = fmax(x - chance(drafter(t), i, dm) / dz, 0.0);
    }
    return x;
  };
  // threads sum consecutive ids
  const int per = (V + kBlock - 1) / kBlock;
  const int i0 = tid * per < V ? tid * per : V, i1 = i0 + per < V ? i0 + per : V;
  double mine = 0, all = 0;
  for (int pass = 0; pass < 2; ++pass) {
    mine = 0;
    for (int i = i0; i < i1; ++i) mine += weight(i);
    all = block_sum(mine, red);
    if (all > 0 || !rest) break;
    rest = false;
  }
  __syncthreads();
  red[tid] = mine;
  __syncthreads();
  if (tid != 0) return;
  const float u = fminf(fmaxf(p.uniforms[(long)n * p.t_max + T_n - 1], 0.f), 1.f);
  const double border = u * all;
  double before = 0;
  int s = 0, last = 0;
  for (int i = 0; i < kBlock; ++i)
    if (red[i] > 0) last = i;
  for (; s < last && before + red[s] <= border; ++s) before += red[s];
  int got = 0;
  for (int i = s * per; i < V && i < (s + 1) * per; ++i) {
    const double x = weight(i);
    if (x > 0) got = i;
    before += x;
    if (x > 0 && before > border) break;
  }
  p.m[n] = m;
  p.next[n] = got;
}

}  // namespace gdnv

extern "C" size_t gdn_draft_verify_workspace_bytes(int32_t n_lanes,
                                                   int32_t t_max,
                                                   int32_t vocab) {
  return 0;
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
  if (n_lanes < 1 || n_lanes > GDN_MAX_LANES || t_max < 1 ||
      t_max > GDN_MAX_T || vocab < 1 || vocab > 1 << 30 || row_stride < vocab ||
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
                 draft_stride, n_lanes, t_max, vocab};
  const dim3 grid((unsigned)n_lanes), block(kBlock);
  const hipError_t e =
      in_dtype == GDN_BF16
          ? launch(verify_kernel<uint16_t>, grid, block, (hipStream_t)stream, p, tl)
          : launch(verify_kernel<float>, grid, block, (hipStream_t)stream, p, tl);
  return gdn::hip_status(e, "gdn_draft_verify launch");
}
