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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// What a slice of a row leaves behind: its largest logit, and Z and W of the
// slice with that as m (W in units of log 2).
struct Part {
  float m, z, w;
  int n;  // alternatives listed
};

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
  int slices;        // slices per row
  Part* parts;       // [rows][slices]
  float* values;     // [rows][slices][n_top]: logits, largest first
  int* ids;          // [rows][slices][n_top]
};

__device__ __forceinline__ float logit_at(const uint16_t* p, long i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}
__device__ __forceinline__ float logit_at(const float* p, long i) {
  return p[i];
}

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

// Larger logits have larger keys; -0 and 0 have the same.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_max(float x) {
  return fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(
                      __float_as_int(-INFINITY), __float_as_int(x), CTRL, ROWS,
                      0xf, false)));
}
// The largest of the 64 lanes' values, in every lane.
__device__ __forceinline__ float wave_max(float x) {
  x = dpp_max<0x111, 0xf>(x);
  x = dpp_max<0x112, 0xf>(x);
  x = dpp_max<0x114, 0xf>(x);
  x = dpp_max<0x118, 0xf>(x);
  x = dpp_max<0x142, 0xa>(x);
  x = dpp_max<0x143, 0xc>(x);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}
__device__ __forceinline__ int wave_prefix(int x) {  // exclusive sum
  int y = x;
  y += __builtin_amdgcn_update_dpp(0, y, 0x111, 0xf, 0xf, false);
  y += __builtin_amdgcn_update_dpp(0, y, 0x112, 0xf, 0xf, false);
  y += __builtin_amdgcn_update_dpp(0, y, 0x114, 0xf, 0xf, false);
  y += __builtin_amdgcn_update_dpp(0, y, 0x118, 0xf, 0xf, false);
  y += __builtin_amdgcn_update_dpp(0, y, 0x142, 0xa, 0xf, false);
  y += __builtin_amdgcn_update_dpp(0, y, 0x143, 0xc, 0xf, false);
  return y - x;
}

// log Z and the row's state from its sums: bad (a NaN or +inf in it), or
// empty (nothing but -inf).
struct RowSums {
  float m, lz, entropy;
  bool bad, empty;
};
__device__ __forceinline__ RowSums row_sums(float m, float z, float w) {
  RowSums r;
  r.bad = !(m < INFINITY) || z != z;
  r.empty = !r.bad && m == -INFINITY;
  r.m = m;
  r.lz = logf(z);
  r.entropy = r.bad ? NAN : r.empty ? 0.f : r.lz - w * kLn2 / z;
  return r;
}
__device__ __forceinline__ float log_p(const ScoreArgs& p, const RowSums& r,
                                       float x) {
  return r.bad ? NAN : r.empty ? -INFINITY : (x - r.m) * p.it - r.lz;
}
template <typename TIn>
__device__ __forceinline__ void write_row(const ScoreArgs& p, long row,
                                          const RowSums& r) {
  if (p.entropy) p.entropy[row] = r.entropy;
  if (p.logprob) {
    const int t = p.tokens[row];
    float lp = 0.f;
    if (t >= p.vocab) lp = NAN;
    else if (t >= 0)
      lp = log_p(p, r, logit_at((const TIn*)p.logits + row * p.stride, t));
    p.logprob[row] = lp;
  }
}
__device__ __forceinline__ void write_top(const ScoreArgs& p, long row,
                                          const RowSums& r, int place,
                                          float x, int id) {
  p.top_ids[row * p.n_top + place] = r.bad ? -1 : id;
  p.top_logprobs[row * p.n_top + place] = log_p(p, r, x);
}

// One workgroup per slice of a row: 16 V bytes a thread, read once into
// registers; everything else works on those.
//
// Alternatives: with n lanes of a wave each holding a logit of at least tau,
// the wave's n-th largest is at least tau too.  So tau, the n-th largest of a
// wave's 64 lane maxima (by a binary search over its key bits, counting
// lanes), rules out nearly every logit; the largest tau of the four waves is
// used.  What is above tau, and of what equals it the n lowest ids of each
// wave, goes to a list in LDS (about n entries, rarely more), whose entries
// then count the ones before them.  Should more be above tau than the list
// holds (its logits would have to sit in a few lanes), the n largest are
// taken one by one.
//
// What bounds it: the read of the row; the exponentials and comparisons come
// to about two thirds of its time.
constexpr int kList = 512;
constexpr int kStrict = kList - 4 * GDN_MAX_TOP;  // room for those above tau

template <typename TIn, int V, bool TOP>
__global__ __launch_bounds__(kThreads) void slice_kernel(ScoreArgs p) {
  constexpr int E = 16 / sizeof(TIn);  // logits per vector
  __shared__ float wave_m[4], wave_tau[4], sums[2][4];
  __shared__ uint32_t list_key[TOP ? kList : 1];
  __shared__ int list_id[TOP ? kList : 1];
  __shared__ int listed;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long row = blockIdx.x / p.slices;
  const int slice = blockIdx.x % p.slices;
  // Vectors are taken from the 16-byte line the row starts in: the ids of
  // the first one may be negative, those of the last may pass the end.
  const TIn* x = (const TIn*)p.logits + row * p.stride;
  const int skew = (int)((uintptr_t)x % 16 / sizeof(TIn));
  const u32x4* line = reinterpret_cast<const u32x4*>(x - skew);
  const int lines = (p.vocab + skew + E - 1) / E;
  const int first = slice * (kThreads * V) + tid;

  u32x4 raw[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = first + c * kThreads;
    raw[c] = line[i < lines ? i : lines - 1];
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int id = (first + c * kThreads) * E - skew;
    if (id < 0 || id > p.vocab - E) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((unsigned)(id + e) >= (unsigned)p.vocab) {
          if constexpr (sizeof(TIn) == 4) raw[c][e] = 0xff800000u;
          else
            raw[c][e / 2] = e & 1 ? (raw[c][e / 2] & 0xffffu) | 0xff800000u
                                  : (raw[c][e / 2] & 0xffff0000u) | 0xff80u;
        }
    }
  }
  auto at = [&](int c, int e) {
    if constexpr (sizeof(TIn) == 4) return __uint_as_float(raw[c][e]);
    else
      return __uint_as_float(e & 1 ? raw[c][e / 2] & 0xffff0000u
                                   : raw[c][e / 2] << 16);
  };
  auto id_of = [&](int c, int e) {
    return (first + c * kThreads) * E - skew + e;
  };

  float own = -INFINITY;
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) own = fmaxf(own, at(c, e));
  const float wm = wave_max(own);
  if (lane == 0) wave_m[wave] = wm;
  if constexpr (TOP) {
    const uint32_t key = key_of(own);
    uint32_t tau = 0;
#pragma unroll
    for (int b = 31; b >= (sizeof(TIn) == 2 ? 16 : 0); --b) {
      const uint32_t t = tau | 1u << b;
      if (__popcll(__ballot(key >= t)) >= p.n_top) tau = t;
    }
    // (the lower key half of a negative bf16 logit is all ones)
    if (sizeof(TIn) == 2 && !(tau >> 31)) tau |= 0xffffu;
    if (lane == 0) wave_tau[wave] = __uint_as_float(tau);
    if (tid == 0) listed = 0;
  }
  __syncthreads();
  const float m =
      fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3]));

  // sums
  {
    const float ref = m == -INFINITY ? 0.f : m, s = p.it * kLog2e;
    float z = 0.f, w = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = (at(c, e) - ref) * s;
        const float q = __builtin_amdgcn_exp2f(d);
        z += q;
        w = __builtin_fmaf(q, fmaxf(d, -1e30f), w);  // 0, not NaN, for -inf
      }
    z = gdn::wave_sum(z);
    w = gdn::wave_sum(w);
    if (lane == 0) {
      sums[0][wave] = z;
      sums[1][wave] = w;
    }
  }

  if constexpr (TOP) {
    uint32_t tau = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t t = __float_as_uint(wave_tau[i]);
      tau = t > tau ? t : tau;
    }
    // keys above tau, and equal to it
    int ties = 0;  // of this wave so far
    const bool some = __any(key_of(own) >= tau);
    if (some) {
#pragma unroll
      for (int c = 0; c < V; ++c) {
        int equal = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t k = key_of(at(c, e));
          equal += k == tau;
          const uint64_t hits = __ballot(k > tau);
          if (hits) {
            int base = 0;
            if (lane == __builtin_ctzll(hits))
              base = atomicAdd(&listed, __popcll(hits));
            base = __builtin_amdgcn_readlane(base, __builtin_ctzll(hits));
            const int slot =
                base + __builtin_amdgcn_mbcnt_hi(
                           (uint32_t)(hits >> 32),
                           __builtin_amdgcn_mbcnt_lo((uint32_t)hits, 0));
            if (k > tau && slot < kStrict) {
              list_key[slot] = k;
              list_id[slot] = id_of(c, e);
            }
          }
        }
        if (ties < p.n_top && __any(equal > 0)) {
          // the n lowest ids of the wave's ties, behind the strict entries
          equal = 0;
#pragma unroll
          for (int e = 0; e < E; ++e)
            equal += key_of(at(c, e)) == tau &&
                     (unsigned)id_of(c, e) < (unsigned)p.vocab;
          int place = ties + wave_prefix(equal);
          ties += __builtin_amdgcn_readlane(place - ties + equal, 63);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (key_of(at(c, e)) == tau &&
                (unsigned)id_of(c, e) < (unsigned)p.vocab) {
              if (place < p.n_top)
                list_id[kStrict + wave * GDN_MAX_TOP + place] = id_of(c, e);
              ++place;
            }
        }
      }
    }
    if (ties > p.n_top) ties = p.n_top;
    for (int i = ties + lane; i < GDN_MAX_TOP; i += 64)
      list_id[kStrict + wave * GDN_MAX_TOP + i] = -1;
    if (lane < GDN_MAX_TOP) list_key[kStrict + wave * GDN_MAX_TOP + lane] = tau;
  }
  __syncthreads();
  const float z = (sums[0][0] + sums[0][1]) + (sums[0][2] + sums[0][3]);
  const float w = (sums[1][0] + sums[1][1]) + (sums[1][2] + sums[1][3]);
  const bool alone = p.slices == 1;
  const long part = row * p.slices + slice;
  const RowSums r = row_sums(m, z, w);
  if (tid == 0) {
    if (alone) write_row<TIn>(p, row, r);
    else p.parts[part] = {m, z, w, 0};
  }
  if constexpr (TOP) {
    auto put = [&](int place, uint32_t key, int id) {
      const float v =
          __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
      if (alone) {
        write_top(p, row, r, place, v, id);
      } else {
        p.values[part * p.n_top + place] = v;
        p.ids[part * p.n_top + place] = id;
      }
    };
    const int strict = listed;
    if (strict <= kStrict) {
      // every entry counts those before it: the strict ones, and if they are
      // fewer than n the ties
      const int span = strict < p.n_top ? kList - kStrict : 0;
      for (int i = tid; i < strict + span; i += kThreads) {
        const int at_i = i < strict ? i : kStrict + i - strict;
        const uint32_t key = list_key[at_i];
        const int id = list_id[at_i];
        if (id < 0) continue;
        int place = 0;
        for (int j = 0; j < strict; ++j) {
          const uint32_t k = list_key[j];
          place += k > key || (k == key && list_id[j] < id);
        }
        if (i >= strict)
          for (int j = kStrict; j < kList; ++j)
            place += (unsigned)list_id[j] < (unsigned)id;
        if (place < p.n_top) put(place, key, id);
      }
    } else {
      uint32_t last = 0xffffffffu;
      int last_id = -1;
      for (int place = 0; place < p.n_top; ++place) {
        uint32_t best = 0;
        int id = INT_MAX;
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t k = key_of(at(c, e));
            const int i = id_of(c, e);
            const bool after = k < last || (k == last && i > last_id);
            if (after && (unsigned)i < (unsigned)p.vocab &&
                (k > best || (k == best && i < id))) {
              best = k;
              id = i;
            }
          }
        __syncthreads();
        list_key[tid] = best;
        list_id[tid] = id;
        __syncthreads();
        for (int j = 0; j < kThreads; ++j)
          if (list_key[j] > best || (list_key[j] == best && list_id[j] < id)) {
            best = list_key[j];
            id = list_id[j];
          }
        last = best;
        last_id = id;
        if (tid == 0) put(place, best, id);
      }
    }
    // a slice of fewer logits than n
    if (!alone && tid == 0) {
      const int from = slice * (kThreads * V) * E - skew;
      const int begin = from < 0 ? 0 : from;
      const int end = from + kThreads * V * E < p.vocab ? from + kThreads * V * E
                                                        : p.vocab;
      const int have = end - begin;
      p.parts[part].n = have < p.n_top ? have : p.n_top;
    }
  }
}

// Joins the slices of a row, one wave each: the sums, then the n largest by
// taking the largest head of the slices' lists n times.  A lane keeps the
// lists of K consecutive slices, so that equal logits are met lowest id
// first.
template <typename TIn>
__global__ __launch_bounds__(64) void join_kernel(ScoreArgs p) {
  const int lane = threadIdx.x;
  const long row = blockIdx.x;
  const Part* parts = p.parts + row * p.slices;
  float m = -INFINITY;
  bool bad = false;
  for (int i = lane; i < p.slices; i += 64) {
    m = fmaxf(m, parts[i].m);
    bad |= parts[i].z != parts[i].z;
  }
  m = wave_max(m);
  float z = 0.f, w = 0.f;
  for (int i = lane; i < p.slices; i += 64) {
    const Part q = parts[i];
    if (q.m == -INFINITY) continue;
    const float d = (q.m - m) * p.it * kLog2e, f = __builtin_amdgcn_exp2f(d);
    z = __builtin_fmaf(f, q.z, z);
    w = __builtin_fmaf(f, __builtin_fmaf(fmaxf(d, -1e30f), q.z, q.w), w);
  }
  z = gdn::wave_sum(z);
  w = gdn::wave_sum(w);
  if (__any(bad)) z = NAN;
  const RowSums r = row_sums(m, z, w);
  if (lane == 0) write_row<TIn>(p, row, r);
  if (p.n_top == 0) return;

  const int K = (p.slices + 63) / 64;
  const float* values = p.values + row * p.slices * p.n_top;
  const int* ids = p.ids + row * p.slices * p.n_top;
  uint32_t last = 0xffffffffu;
  int last_id = -1;
  // heads of the lane's lists: what comes after (last, last_id) in each
  uint32_t key = 0;  // 0: none left
  float value = 0.f;
  int id = 0, from = 0, taken = 0;
  auto head = [&]() {
    key = 0;
    for (int k = 0; k < K; ++k) {
      const int s = lane * K + k;
      if (s >= p.slices) break;
      const int n = parts[s].n;
      for (int i = K == 1 ? taken : 0; i < n; ++i) {
        const float v = values[(long)s * p.n_top + i];
        const uint32_t q = key_of(v);
        const int j = ids[(long)s * p.n_top + i];
        if (q > last || (q == last && j <= last_id)) continue;
        if (q > key) {
          key = q;
          value = v;
          id = j;
          from = s;
        }
        break;
      }
    }
  };
  head();
  for (int place = 0; place < p.n_top; ++place) {
    uint32_t best = key;
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
      const uint32_t o = __shfl_xor(best, x);
      best = o > best ? o : best;
    }
    const int win = __builtin_ctzll(__ballot(key == best));
    last = best;
    last_id = __shfl(id, win);
    if (lane == win) {
      write_top(p, row, r, place, value, id);
      ++taken;
      head();
    }
  }
}

static bool sizes_ok(int32_t n_rows, int32_t vocab, int32_t n_top) {
  return n_rows >= 1 && vocab >= 1 && n_top >= 0 && n_top <= GDN_MAX_TOP &&
         n_top <= vocab;
}

// Vectors per thread of a slice: eight, or two when eight would leave most
// of the CUs without a slice.
static int vectors_for(int32_t n_rows, int32_t vocab, int size) {
  const long per = (long)kThreads * 8 * 16 / size;
  return n_rows * ((vocab + per - 1) / per) < 256 ? 2 : 8;
}
// (one more vector than the vocabulary fills: rows may start inside one)
static int slices_for(int32_t vocab, int size, int v) {
  const int per_line = 16 / size;
  const long lines = ((long)vocab + per_line - 1) / per_line + 1;
  return (int)((lines + kThreads * v - 1) / (kThreads * v));
}
static size_t round16(size_t n) { return (n + 15) / 16 * 16; }
static size_t bytes_for(int32_t n_rows, int slices, int32_t n_top) {
  const size_t n = (size_t)n_rows * slices;
  return slices == 1 ? 0 : round16(n * sizeof(Part)) + 2 * round16(n * n_top * 4);
}

template <typename TIn>
static hipError_t run(const ScoreArgs& p, int v, hipStream_t st) {
  const dim3 grid((unsigned)((long)p.rows * p.slices)), block(kThreads);
  const bool top = p.n_top > 0;
  hipError_t e;
  if (v == 8)
    e = top ? launch(slice_kernel<TIn, 8, true>, grid, block, st, p)
            : launch(slice_kernel<TIn, 8, false>, grid, block, st, p);
  else
    e = top ? launch(slice_kernel<TIn, 2, true>, grid, block, st, p)
            : launch(slice_kernel<TIn, 2, false>, grid, block, st, p);
  if (e != hipSuccess || p.slices == 1) return e;
  return launch(join_kernel<TIn>, dim3((unsigned)p.rows), dim3(64), st, p);
}

}  // namespace gdnt

extern "C" size_t gdn_token_scores_workspace_bytes(int32_t n_rows,
                                                   int32_t vocab,
                                                   int32_t n_top) {
  using namespace gdnt;
  if (!sizes_ok(n_rows, vocab, n_top)) return 0;
  // the larger of the two types' needs
  size_t need = 0;
  for (int size = 2; size <= 4; size += 2) {
    const int v = vectors_for(n_rows, vocab, size);
    const size_t n = bytes_for(n_rows, slices_for(vocab, size, v), n_top);
    if (n > need) need = n;
  }
  return need;
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
  const int size = in_dtype == GDN_BF16 ? 2 : 4;
  const int v = vectors_for(n_rows, vocab, size);
  ScoreArgs p = {logits, tokens, logprob, entropy, top_ids, top_logprobs,
                 row_stride, n_rows, vocab, n_top, inv_temperature,
                 slices_for(vocab, size, v), nullptr, nullptr, nullptr};
  if ((double)n_rows * p.slices > (double)INT_MAX)
    return fail(GDN_EINVAL, "gdn_token_scores: grid too large");
  const size_t n = (size_t)n_rows * p.slices;
  p.parts = (Part*)workspace;
  p.values = (float*)((char*)workspace + round16(n * sizeof(Part)));
  p.ids = (int*)((char*)p.values + round16(n * n_top * 4));
  const hipError_t e = in_dtype == GDN_BF16
                           ? run<uint16_t>(p, v, (hipStream_t)stream)
                           : run<float>(p, v, (hipStream_t)stream);
  return gdn::hip_status(e, "gdn_token_scores launch");
}
