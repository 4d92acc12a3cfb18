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

#include <cfloat>
#include <cmath>

#include "gdn.h"
#include "gdn_window_common.h"

namespace gdnt {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// What a slice of a row leaves behind: its largest logit, and Z and W of the
// slice with that as m (W in units of the logits).
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
__device__ __forceinline__ RowSums row_sums(float m, float z, float w,
                                            float it) {
  RowSums r;
  r.bad = !(m < INFINITY) || z != z;
  r.empty = !r.bad && m == -INFINITY;
  r.m = m;
  r.lz = logf(z);
  r.entropy = r.bad ? NAN : r.empty ? 0.f : r.lz - w * it / z;
  return r;
}
__device__ __forceinline__ float log_p(const ScoreArgs& p, const RowSums& r,
                                       float x) {
  // (halves: the difference of two logits may be past f32 where its product
  // with a small inverse temperature is not)
  return r.bad     ? NAN
         : r.empty ? -INFINITY
                   : (0.5f * x - 0.5f * r.m) * (2.f * p.it) - r.lz;
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

constexpr int kList = 512;
constexpr int kStrict = kList - 4 * GDN_MAX_TOP;  // room for those above tau

// Whether a row's slices, of N logits per thread at most, are equally long: a
// short last one has few threads with logits, and then the alternatives take
// the slow way (53 rows x 2214 logits, top 20: 20 -> 14 us).  Slices of many
// logits are full, which keeps their ids simple (108 -> 75 us for 1024 rows x
// 131,072).
template <int N>
constexpr bool kEven = N == 8;

// The n largest of a slice when more than the list holds is at least tau (or
// tau is -inf, where entries that stand for no logit look the same).
template <typename TIn, int V, typename Put>
__device__ __forceinline__ void pick_tied(
    const ScoreArgs& p, const float (&val)[V][16 / sizeof(TIn)], uint32_t tau,
    int first, int end, int skew, int& listed, uint32_t* list_key,
    int* list_id, Put&& put) {
  constexpr int E = 16 / sizeof(TIn);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto id_of = [&](int c, int e) {
    const int i = first + c * kThreads;
    // (no id behind the end of an even slice; other slices end with the row)
    return kEven<V * E> && i >= end ? -1 : i * E - skew + e;
  };
  __syncthreads();
  if (tid == 0) listed = 0;
  __syncthreads();
  int ties = 0;  // of this wave so far
#pragma unroll
  for (int c = 0; c < V; ++c) {
    int equal = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t k = key_of(val[c][e]);
      if (k > tau) {
        const int slot = atomicAdd(&listed, 1);
        if (slot < kStrict) {
          list_key[slot] = k;
          list_id[slot] = id_of(c, e);
        }
      }
      equal += k == tau && (unsigned)id_of(c, e) < (unsigned)p.vocab;
    }
    if (ties < p.n_top && __any(equal > 0)) {
      // the n lowest ids of the wave's ties, behind the entries above tau
      int place = ties + wave_prefix(equal);
      ties = __builtin_amdgcn_readlane(place + equal, 63);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (key_of(val[c][e]) == tau &&
            (unsigned)id_of(c, e) < (unsigned)p.vocab) {
          if (place < p.n_top)
            list_id[kStrict + wave * GDN_MAX_TOP + place] = id_of(c, e);
          ++place;
        }
    }
  }
  for (int i = ties + lane; i < GDN_MAX_TOP; i += 64)
    list_id[kStrict + wave * GDN_MAX_TOP + i] = -1;
  if (lane < GDN_MAX_TOP) {
    list_key[kStrict + wave * GDN_MAX_TOP + lane] = tau;
    if (lane >= p.n_top) list_id[kStrict + wave * GDN_MAX_TOP + lane] = -1;
  }
  __syncthreads();
  const int strict = listed;
  if (strict <= kStrict) {
    // every entry counts those before it: the ones above tau, and if they
    // are fewer than n the ties
    const int span = strict < p.n_top ? kList - kStrict : 0;
    for (int i = tid; i < strict + span; i += kThreads) {
      const int at_i = i < strict ? i : kStrict + i - strict;
      const uint32_t key = list_key[at_i];
      const int id = list_id[at_i];
      if (id < 0) continue;
      int place = 0;
#pragma unroll 4
      for (int j = 0; j < strict; ++j) {
        const uint32_t k = list_key[j];
        place += k > key || (k == key && list_id[j] < id);
      }
      if (i >= strict)
#pragma unroll 4
        for (int j = kStrict; j < kList; ++j)
          place += (unsigned)list_id[j] < (unsigned)id;
      if (place < p.n_top) put(place, key, id);
    }
    return;
  }
  uint32_t last = 0xffffffffu;
  int last_id = -1;
  for (int place = 0; place < p.n_top; ++place) {
    uint32_t best = 0;
    int id = INT_MAX;
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t k = key_of(val[c][e]);
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
#pragma unroll 4
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

// One workgroup per slice of a row: 16 V bytes a thread, read once into
// registers; everything else works on those.
//
// Alternatives: with n threads each holding a logit of at least tau, the n-th
// largest of the slice is at least tau too.  So tau, the n-th largest of the
// 256 thread maxima cut to the upper half of its key (by a binary search over
// those bits, counting threads; every wave for itself), rules out nearly every
// logit.  What is at least tau goes to a list in LDS (about n entries, rarely
// more), whose entries then count the ones before them.  If that is more than
// the list holds (many equal logits), what is above tau and, of what equals
// it, the n lowest ids of each wave are listed instead; and if even what is
// above tau is too much (it would have to sit in a few lanes), the n largest
// are taken one by one.
//
// Bound by vector instructions, about nine per logit for the sums and a
// quarter of its time for the alternatives: 1024 rows x 131,072 bf16 logits,
// top 20, in 76 us (3.6 TB/s) with the vector ALUs issuing in every cycle; 16
// f32 rows in 6.5 us.  (64 logits a thread
// took too many registers, 269 us; a tau per wave instead of per workgroup
// left four times the entries, 190 us.)
template <typename TIn, int V, bool TOP>
__global__ __launch_bounds__(kThreads, 4) void slice_kernel(ScoreArgs p) {
  constexpr int E = 16 / sizeof(TIn);  // logits per vector
  __shared__ __attribute__((aligned(16))) float own_of[kThreads];
  __shared__ float sums[2][4];
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
  const int per = kEven<V * E> ? (lines + p.slices - 1) / p.slices : kThreads * V;
  const int first = slice * per + tid;
  const int end = (slice + 1) * per < lines ? (slice + 1) * per : lines;

  u32x4 raw[V];
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = first + c * kThreads;
    raw[c] = line[i < end ? i : lines - 1];
  }
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int i = first + c * kThreads, id = i < end ? i * E - skew : p.vocab;
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
  float val[V][E];
#pragma unroll
  for (int c = 0; c < V; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if constexpr (sizeof(TIn) == 4) val[c][e] = __uint_as_float(raw[c][e]);
      else
        val[c][e] = __uint_as_float(e & 1 ? raw[c][e / 2] & 0xffff0000u
                                          : raw[c][e / 2] << 16);
  auto id_of = [&](int c, int e) {
    return (first + c * kThreads) * E - skew + e;
  };

  float top[V], own = -INFINITY;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    top[c] = val[c][0];
#pragma unroll
    for (int e = 1; e < E; ++e) top[c] = fmaxf(top[c], val[c][e]);
    own = fmaxf(own, top[c]);
  }
  own_of[tid] = own;
  if (TOP && tid == 0) listed = 0;
  __syncthreads();
  const f32x4 of4 = *reinterpret_cast<const f32x4*>(&own_of[4 * lane]);
  const float m =
      wave_max(fmaxf(fmaxf(of4[0], of4[1]), fmaxf(of4[2], of4[3])));
  uint32_t keys[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) keys[i] = key_of(of4[i]);
  auto search = [&](uint32_t tau, int from, int to) {
    for (int b = from; b >= to; --b) {
      const uint32_t t = tau | 1u << b;
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += __popcll(__ballot(keys[i] >= t));
      if (n >= p.n_top) tau = t;
    }
    return tau;
  };

  // sums (W in units of the logits)
  {
    const float ref = m == -INFINITY ? 0.f : m, s = p.it * kLog2e;
    float z = 0.f, w = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // (0 times the d of a -inf has to be 0; a NaN stays one)
        const float d =
            __builtin_elementwise_maximum(val[c][e] - ref, -FLT_MAX);
        const float q = __builtin_amdgcn_exp2f(d * s);
        z += q;
        w = __builtin_fmaf(q, d, w);
      }
    z = gdn::wave_sum(z);
    w = gdn::wave_sum(w);
    if (lane == 0) {
      sums[0][wave] = z;
      sums[1][wave] = w;
    }
  }

  uint32_t tau = 0;
  if constexpr (TOP) {
    tau = search(0, 31, 16);
    const float least = __uint_as_float(tau >> 31 ? tau & 0x7fffffffu : ~tau);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if (top[c] >= least) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (val[c][e] >= least) {
            const int slot = atomicAdd(&listed, 1);
            if (slot < kList) {
              list_key[slot] = key_of(val[c][e]);
              list_id[slot] = id_of(c, e);
            }
          }
      }
    }
  }
  __syncthreads();
  const float z = (sums[0][0] + sums[0][1]) + (sums[0][2] + sums[0][3]);
  const float w = (sums[1][0] + sums[1][1]) + (sums[1][2] + sums[1][3]);
  const bool alone = p.slices == 1;
  const long part = row * p.slices + slice;
  const RowSums r = row_sums(m, z, w, p.it);
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
    const int entries = listed;
    const int begin = slice == 0 ? 0 : slice * per * E - skew;
    const int stop = end * E - skew < p.vocab ? end * E - skew : p.vocab;
    const int have = stop - begin < 0 ? 0 : stop - begin;
    const int wanted = have < p.n_top ? have : p.n_top;
    if (alone && r.bad) {  // (a negative NaN is in none of the lists)
      if (tid < p.n_top) write_top(p, row, r, tid, 0.f, -1);
    } else if (m == -INFINITY) {  // nothing but -inf: the lowest ids
      if (tid < wanted) put(tid, key_of(-INFINITY), begin + tid);
    } else if (entries <= kList && tau > key_of(-INFINITY)) {
      for (int i = tid; i < entries; i += kThreads) {
        const uint32_t key = list_key[i];
        const int id = list_id[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < entries; ++j) {
          const uint32_t k = list_key[j];
          place += k > key || (k == key && list_id[j] < id);
        }
        if (place < p.n_top) put(place, key, id);
      }
    } else {
      tau = search(tau, 15, 0);
      pick_tied<TIn, V>(p, val, tau, first, end, skew, listed, list_key, list_id,
                        put);
    }
    if (!alone && tid == 0) p.parts[part].n = wanted;
  }
}

// Joins the slices of a row: the sums (every wave for itself), then as in a
// slice: with tau at most the n-th largest of 256 sampled entries, the first
// ones of every list, what is at least tau goes to a list in LDS (a little
// more than n entries), whose entries count the ones before them.  Should
// they not fit (equal logits in many slices), the first wave takes the largest
// head of the lists n times; a lane keeps the lists of K consecutive slices,
// so that equal logits are met lowest id first.
// Bound by its launch and three loads in a row: 9 us for 1024 rows of 16 lists
// of 20, 5 us for 16 rows.  (Taking the largest head of the lists n times from
// the start took 11 and 5 us, and 9 to 16 us for few rows of lists of 20 to
// 32, now 6 to 8.)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max_key(uint32_t x) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL,
                                                           ROWS, 0xf, false);
  return o > x ? o : x;
}
__device__ __forceinline__ uint32_t wave_max_key(uint32_t x) {
  x = dpp_max_key<0x111, 0xf>(x);
  x = dpp_max_key<0x112, 0xf>(x);
  x = dpp_max_key<0x114, 0xf>(x);
  x = dpp_max_key<0x118, 0xf>(x);
  x = dpp_max_key<0x142, 0xa>(x);
  x = dpp_max_key<0x143, 0xc>(x);
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

template <typename TIn, bool TOP>
__global__ __launch_bounds__(TOP ? kThreads : 64) void join_kernel(ScoreArgs p) {
  __shared__ __attribute__((aligned(16))) uint32_t sample_of[kThreads];
  __shared__ uint32_t list_key[TOP ? kList : 1];
  __shared__ int list_id[TOP ? kList : 1];
  __shared__ int listed;
  const int tid = threadIdx.x, lane = tid & 63;
  const long row = blockIdx.x;
  const Part* parts = p.parts + row * p.slices;
  const int all = p.slices * p.n_top;
  const float* values = p.values + row * all;
  const int* ids = p.ids + row * all;
  uint32_t sample = 0;  // (below every key)
  if constexpr (TOP) {
    if (p.slices <= kThreads) {
      const int s = tid % p.slices, i = tid / p.slices;
      if (i < p.n_top && i < parts[s].n)
        sample = key_of(values[s * p.n_top + i]);
    } else {
      for (int s = tid; s < p.slices; s += kThreads)
        if (parts[s].n > 0) {
          const uint32_t k = key_of(values[s * p.n_top]);
          sample = k > sample ? k : sample;
        }
    }
    sample_of[tid] = sample;
    if (tid == 0) listed = 0;
  }
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
    const float d = q.m - m, f = __builtin_amdgcn_exp2f(d * (p.it * kLog2e));
    if (f == 0.f) continue;  // (d z may have left f32: a slice of lowest values)
    z = __builtin_fmaf(f, q.z, z);
    w = __builtin_fmaf(f, __builtin_fmaf(d, q.z, q.w), w);
  }
  z = gdn::wave_sum(z);
  w = gdn::wave_sum(w);
  if (__any(bad)) z = NAN;
  const RowSums r = row_sums(m, z, w, p.it);
  if (tid == 0) write_row<TIn>(p, row, r);
  if constexpr (TOP) {
    if (r.bad) {  // (the lists may lack entries)
      if (tid < p.n_top) write_top(p, row, r, tid, 0.f, -1);
      return;
    }
    __syncthreads();
    const u32x4 of4 = *reinterpret_cast<const u32x4*>(&sample_of[4 * lane]);
    uint32_t tau = 0;
    for (int b = 31; b >= 16; --b) {
      const uint32_t t = tau | 1u << b;
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += __popcll(__ballot(of4[i] >= t));
      if (n >= p.n_top) tau = t;
    }
    for (int i = tid; i < all; i += kThreads) {
      const uint32_t key = key_of(values[i]);
      if (key < tau) continue;
      const int s = i / p.n_top;
      if (i - s * p.n_top >= parts[s].n) continue;
      const int slot = atomicAdd(&listed, 1);
      if (slot < kList) {
        list_key[slot] = key;
        list_id[slot] = ids[i];
      }
    }
    __syncthreads();
    const int entries = listed;
    if (entries <= kList) {
      for (int i = tid; i < entries; i += kThreads) {
        const uint32_t key = list_key[i];
        const int id = list_id[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < entries; ++j) {
          const uint32_t k = list_key[j];
          place += k > key || (k == key && list_id[j] < id);
        }
        if (place < p.n_top)
          write_top(p, row, r, place,
                    __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key), id);
      }
      return;
    }
    if (tid >= 64) return;
    const int K = (p.slices + 63) / 64;
    uint32_t last = 0xffffffffu;
    int last_id = -1;
    // head of the lane's lists: the first of what comes after (last, last_id)
    uint32_t key = 0;  // 0: none left
    float value = 0.f;
    int id = 0;
    auto head = [&]() {
      key = 0;
      for (int k = 0; k < K; ++k) {
        const int s = lane * K + k;
        if (s >= p.slices) break;
        const int n = parts[s].n;
        for (int i = 0; i < n; ++i) {
          const float v = values[s * p.n_top + i];
          const uint32_t q = key_of(v);
          const int j = ids[s * p.n_top + i];
          if (q > last || (q == last && j <= last_id)) continue;
          if (q > key) {
            key = q;
            value = v;
            id = j;
          }
          break;
        }
      }
    };
    head();
    for (int place = 0; place < p.n_top; ++place) {
      const uint32_t best = wave_max_key(key);
      const int win = __builtin_ctzll(__ballot(key == best));
      last = best;
      last_id = __builtin_amdgcn_readlane(id, win);
      if (lane == win) {
        write_top(p, row, r, place, value, id);
        head();
      }
    }
  }
}

static bool sizes_ok(int32_t n_rows, int32_t vocab, int32_t n_top) {
  return n_rows >= 1 && vocab >= 1 && vocab <= 1 << 30 && n_top >= 0 && n_top <= GDN_MAX_TOP &&
         n_top <= vocab;
}

// Vectors per thread of a slice: 32 logits a thread, or 8 when that would
// leave most of the CUs without a slice.
static int vectors_for(int32_t n_rows, int32_t vocab, int size) {
  const long per = (long)kThreads * 32;
  return (n_rows * ((vocab + per - 1) / per) < 256 ? 8 : 32) * size / 16;
}
// aligned: every row starts with a vector; else it may reach into one more
// than it fills.
static int slices_for(int32_t vocab, int size, int v, bool aligned) {
  const int per_line = 16 / size;
  const long lines = ((long)vocab + per_line - 1) / per_line + (aligned ? 0 : 1);
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
  constexpr int kMany = 32 * sizeof(TIn) / 16, kFew = 8 * sizeof(TIn) / 16;
  if (v == kMany)
    e = top ? launch(slice_kernel<TIn, kMany, true>, grid, block, st, p)
            : launch(slice_kernel<TIn, kMany, false>, grid, block, st, p);
  else
    e = top ? launch(slice_kernel<TIn, kFew, true>, grid, block, st, p)
            : launch(slice_kernel<TIn, kFew, false>, grid, block, st, p);
  if (e != hipSuccess || p.slices == 1) return e;
  const dim3 rows((unsigned)p.rows);
  return top ? launch(join_kernel<TIn, true>, rows, block, st, p)
             : launch(join_kernel<TIn, false>, rows, dim3(64), st, p);
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
    const size_t n = bytes_for(n_rows, slices_for(vocab, size, v, false), n_top);
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
  if (!(inv_temperature >= 1e-30f) || !(inv_temperature <= 1e30f))
    return fail(GDN_EINVAL,
                "gdn_token_scores: inv_temperature out of 1e-30..1e30");
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
                 slices_for(vocab, size, v,
                            !misaligned(logits, 16) &&
                                (n_rows == 1 || row_stride * size % 16 == 0)),
                 nullptr, nullptr, nullptr};
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
