// gdn_scores.h -- log probabilities of given tokens, entropies and top
// alternatives of rows of logits (gdn_token_scores).  Compiled as part of
// gdn_state.hip.
//
// With x = inv_temperature * logit, m = max x, e_i = exp(x_i - m),
// Z = sum e_i and W = sum e_i (x_i - m):
//   log p_i = x_i - m - log Z,   entropy = log Z - W / Z.
// The order of the alternatives is that of the logits themselves (larger
// first, equal ones by the lower id), which scaling keeps.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_window_common.h"

namespace gdnt {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;

struct ScoreArgs {
  const void* logits;
  const int* tokens;
  float* logprob;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  long stride;
  int rows, vocab, n_top;
  float it;
};

__device__ __forceinline__ float logit_at(const uint16_t* p, long i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}
__device__ __forceinline__ float logit_at(const float* p, long i) {
  return p[i];
}

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float x, float* buf) {
  x = gdn::wave_sum(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x / 64] = x;
  __syncthreads();
  return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

// One workgroup per row, a pass over the row for every quantity.
template <typename TIn>
__global__ __launch_bounds__(kThreads) void scores_kernel(ScoreArgs p) {
  __shared__ float buf[4];
  __shared__ float bv[kThreads];
  __shared__ int bi[kThreads];
  const int tid = threadIdx.x;
  const long row = blockIdx.x;
  const TIn* x = (const TIn*)p.logits + row * p.stride;
  float m = -INFINITY;
  int bad = 0;
  for (int i = tid; i < p.vocab; i += kThreads) {
    const float v = logit_at(x, i);
    bad |= !(v < INFINITY);
    m = fmaxf(m, v);
  }
  bad = __syncthreads_or(bad);
  bv[tid] = m;
  __syncthreads();
  for (int s = kThreads / 2; s > 0; s >>= 1) {
    if (tid < s) bv[tid] = fmaxf(bv[tid], bv[tid + s]);
    __syncthreads();
  }
  m = bv[0];
  __syncthreads();
  const bool empty = !bad && m == -INFINITY;
  float z = 0.f, w = 0.f;
  if (!bad && !empty) {
    for (int i = tid; i < p.vocab; i += kThreads) {
      const float d = (logit_at(x, i) - m) * p.it;
      const float e = expf(d);
      z += e;
      if (e > 0.f) w = __builtin_fmaf(e, d, w);
    }
  }
  z = block_sum(z, buf);
  w = block_sum(w, buf);
  const float lz = logf(z);
  if (tid == 0) {
    if (p.entropy) p.entropy[row] = bad ? NAN : empty ? 0.f : lz - w / z;
    if (p.logprob) {
      const int t = p.tokens[row];
      float lp;
      if (t < 0) lp = 0.f;
      else if (bad || t >= p.vocab) lp = NAN;
      else if (empty) lp = -INFINITY;
      else lp = (logit_at(x, t) - m) * p.it - lz;
      p.logprob[row] = lp;
    }
  }
  float last = INFINITY;
  int last_id = -1;
  for (int j = 0; j < p.n_top; ++j) {
    if (bad) {
      if (tid == 0) {
        p.top_ids[row * p.n_top + j] = -1;
        p.top_logprobs[row * p.n_top + j] = NAN;
      }
      continue;
    }
    // the largest entry after (last, last_id) in the order
    float best = -INFINITY;
    int id = INT_MAX;
    for (int i = tid; i < p.vocab; i += kThreads) {
      const float v = logit_at(x, i);
      const bool after = v < last || (v == last && i > last_id);
      if (after && (v > best || (v == best && i < id))) {
        best = v;
        id = i;
      }
    }
    bv[tid] = best;
    bi[tid] = id;
    __syncthreads();
    for (int s = kThreads / 2; s > 0; s >>= 1) {
      if (tid < s) {
        const float v = bv[tid + s];
        const int i = bi[tid + s];
        if (v > bv[tid] || (v == bv[tid] && i < bi[tid])) {
          bv[tid] = v;
          bi[tid] = i;
        }
      }
      __syncthreads();
    }
    last = bv[0];
    last_id = bi[0];
    __syncthreads();
    if (tid == 0) {
      p.top_ids[row * p.n_top + j] = last_id;
      p.top_logprobs[row * p.n_top + j] =
          empty ? -INFINITY : (last - m) * p.it - lz;
    }
  }
}

static bool sizes_ok(int32_t n_rows, int32_t vocab, int32_t n_top) {
  return n_rows >= 1 && vocab >= 1 && n_top >= 0 && n_top <= GDN_MAX_TOP &&
         n_top <= vocab;
}

}  // namespace gdnt

extern "C" size_t gdn_token_scores_workspace_bytes(int32_t n_rows,
                                                   int32_t vocab,
                                                   int32_t n_top) {
  if (!gdnt::sizes_ok(n_rows, vocab, n_top)) return 0;
  return 0;
}

extern "C" int gdn_token_scores(int32_t n_rows, int32_t vocab,
                                int64_t row_stride, const void* logits,
                                int in_dtype, const int32_t* tokens,
                                int32_t n_top, float inv_temperature,
                                float* logprob, float* entropy,
                                int32_t* top_ids, float* top_logprobs,
                                void* workspace, size_t ws_bytes,
                                void* stream) {
  using namespace gdnt;
  if (!sizes_ok(n_rows, vocab, n_top) || row_stride < vocab)
    return fail(GDN_EINVAL, "gdn_token_scores: sizes out of range");
  if (in_dtype != GDN_BF16 && in_dtype != GDN_F32)
    return fail(GDN_EINVAL, "gdn_token_scores: unknown in_dtype");
  if (!(inv_temperature > 0.f) || !(inv_temperature < INFINITY))
    return fail(GDN_EINVAL,
                "gdn_token_scores: inv_temperature must be finite and > 0");
  if (!logits || (tokens && !logprob) || (!tokens && logprob) ||
      (n_top > 0 && (!top_ids || !top_logprobs)))
    return fail(GDN_EINVAL, "gdn_token_scores: required pointer is NULL");
  if (!logprob && !entropy && n_top == 0)
    return fail(GDN_EINVAL, "gdn_token_scores: no output is wanted");
  if (misaligned(logits, in_dtype == GDN_BF16 ? 2 : 4) ||
      misaligned(tokens, 4) || misaligned(logprob, 4) ||
      misaligned(entropy, 4) || misaligned(top_ids, 4) ||
      misaligned(top_logprobs, 4) || misaligned(workspace, 16))
    return fail(GDN_EINVAL, "gdn_token_scores: misaligned pointer");
  const size_t need = gdn_token_scores_workspace_bytes(n_rows, vocab, n_top);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_token_scores: workspace too small");
  const ScoreArgs p = {logits,      tokens,       logprob,
                       entropy,     top_ids,      top_logprobs,
                       row_stride,  n_rows,       vocab,
                       n_top,       inv_temperature};
  const dim3 grid((unsigned)n_rows), block(kThreads);
  const hipError_t e =
      in_dtype == GDN_BF16
          ? launch(scores_kernel<uint16_t>, grid, block, (hipStream_t)stream, p)
          : launch(scores_kernel<float>, grid, block, (hipStream_t)stream, p);
  return gdn::hip_status(e, "gdn_token_scores launch");
}
