// gdn_rope.h -- the writer of the paged cache with the position rotation on
// the way (gdn_rope_append, gdn_rope_append_mxfp).  Compiled as part of
// gdn_state.hip.
//
// Channel pair (a, b) of a query or key row at position p turns by the angle
// p f_i (f_i the pair's inverse frequency):
//   a' = a cos - b sin,   b' = b cos + a sin.
// p f_i has at most 31 + 24 significant bits, so its product in f64 is exact
// to half a step (for positions below 2^29 altogether), and it is reduced to a
// fraction of a turn there: the angle is as good at the far end of a long cache
// as at its start.
//
// Every row is read and written once; memory bounds a large call, the launch
// and what the caller does for it a small one (3.3 us of kernel for 8 lanes
// of one token, 18 heads of 256; 4.5 into 4 bits).  128 lanes x 64 tokens, 48
// heads of 128, bf16: 47 us, 201 MB at 4.3 TB/s, a large copy runs at 4.6 to 4.8;
// the same into 4 bits, the decoded rows written as well: 48 us, 211 MB at 4.4
// (with keys turned in f32, see code_rows, 1.3 us less).
// What it took: a thread that turns one head works out eight angles in f64
// for it, 102 and 107 us; with the angles kept for the same channels of
// several heads (see slots_for) they cost nothing.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_mxfp.h"
#include "gdn_paged.h"

namespace gdnk {

struct RopeArgs {
  KvArgs kv;  // k, v: the caches (rows in their type) or unused
  const void *q, *k, *v;
  long qs, ks, vs;  // elements from a token's rows to the next token's
  void* q_out;
  void *kc, *vc;         // caches, or
  Fp4Rows k4, v4;        // the 4-bit caches
  uint16_t *k_held, *v_held;
  const float* inv_freq;
  const int* positions;
  int rot;
  bool pairs;  // neighbouring channels form pairs, else channels rot / 2 apart
};

// An angle p f as quarter turns and a rest x of at most an eighth of a turn.
__device__ __forceinline__ int reduced(int p, float f, double& x) {
  const double a = (double)p * (double)f;
  // 1 / (2 pi) in two parts
  constexpr double kHi = 0.15915494309189534561, kLo = -9.8393383375912e-18;
  const double whole = __builtin_rint(a * kHi);
  const double r =
      __builtin_fma(a, kHi, -whole) + a * kLo;  // -1/2 .. 1/2
  const double quarter = __builtin_rint(4.0 * r);
  x = (r - 0.25 * quarter) * 6.28318530717958647693;
  return (int)quarter & 3;
}
// Cosine and sine of x and k quarter turns from those of x.
template <typename F>
__device__ __forceinline__ void turned(int k, F cs, F sn, F& c, F& s) {
  const F u = k & 1 ? sn : cs, v = k & 1 ? cs : sn;
  c = k == 1 || k == 2 ? -u : u;
  s = k >= 2 ? -v : v;
}
// cos and sin of p f in f32: Taylor series whose next terms are below 2^-25 at
// pi / 4.
__device__ __forceinline__ void turn(int p, float f, float& c, float& s) {
  double rest;
  const int k = reduced(p, f, rest);
  const float x = (float)rest, y = x * x;
  float sn = __builtin_fmaf(y, 2.75573192e-6f, -1.98412698e-4f);
  sn = __builtin_fmaf(y, sn, 8.33333333e-3f);
  sn = __builtin_fmaf(y, sn, -1.66666667e-1f);
  sn = __builtin_fmaf(x * y, sn, x);
  float cs = __builtin_fmaf(y, -2.75573192e-7f, 2.48015873e-5f);
  cs = __builtin_fmaf(y, cs, -1.38888889e-3f);
  cs = __builtin_fmaf(y, cs, 4.16666667e-2f);
  cs = __builtin_fmaf(y, cs, -0.5f);
  cs = __builtin_fmaf(y, cs, 1.f);
  turned(k, cs, sn, c, s);
}
// The same in f64, the next terms 2e-14 and 1e-15 at pi / 4.
__device__ __forceinline__ void turn(int p, float f, double& c, double& s) {
  double x;
  const int k = reduced(p, f, x);
  const double y = x * x;
  double sn = __builtin_fma(y, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  sn = __builtin_fma(y, sn, 1.0 / 362880.0);
  sn = __builtin_fma(y, sn, -1.0 / 5040.0);
  sn = __builtin_fma(y, sn, 1.0 / 120.0);
  sn = __builtin_fma(y, sn, -1.0 / 6.0);
  sn = __builtin_fma(x * y, sn, x);
  double cs = __builtin_fma(y, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  cs = __builtin_fma(y, cs, -1.0 / 3628800.0);
  cs = __builtin_fma(y, cs, 1.0 / 40320.0);
  cs = __builtin_fma(y, cs, -1.0 / 720.0);
  cs = __builtin_fma(y, cs, 1.0 / 24.0);
  cs = __builtin_fma(y, cs, -0.5);
  cs = __builtin_fma(y, cs, 1.0);
  turned(k, cs, sn, c, s);
}

// Eight channels of a row.
struct Eight {
  float x[8];
};
__device__ __forceinline__ Eight load_eight(const uint16_t* p) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = __uint_as_float(w[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Eight load_eight(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
  const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
  return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ void store_eight(uint16_t* p, const Eight& r) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf16_pair(r.x[2 * i], r.x[2 * i + 1]);
  *reinterpret_cast<u32x4*>(p) = w;
}
__device__ __forceinline__ void store_eight(float* p, const Eight& r) {
  *reinterpret_cast<f32x4*>(p) = f32x4{r.x[0], r.x[1], r.x[2], r.x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{r.x[4], r.x[5], r.x[6], r.x[7]};
}
// Position of token t of lane n in the cache (-1: none) and for the rotation.
__device__ __forceinline__ int slot_of(const KvArgs& a, int n, int t, int T) {
  const long pos = (long)a.kv_len[n] - T + t;
  return pos < 0 || pos >= a.max_pages * a.page ? -1 : (int)pos;
}
__device__ __forceinline__ int turn_of(const RopeArgs& p, int n, int t, int T) {
  return p.positions ? p.positions[(long)n * p.kv.t_max + t]
                     : (int)((unsigned)p.kv.kv_len[n] - T + t);
}

// Cosines and sines of N pairs from inverse frequency f on.
template <int N, typename F = float>
struct Turns {
  F c[N], s[N];
  __device__ __forceinline__ void set(int pos, const float* f) {
#pragma unroll
    for (int i = 0; i < N; ++i) turn(pos, f[i], c[i], s[i]);
  }
};

// How a launch is shared out: blocks of threads that turn rows (a thread takes
// the same channels of every `slots`-th head, so that it works out its angles
// once), then blocks that copy, then blocks that write 4-bit rows.
struct RopePlan {
  int units, slots, heads, blocks;  // turning: units and heads of a token
  int pieces, copy_blocks;          // copying: 16-byte pieces of a token
  int slots4;                       // 4-bit rows: as slots
};
constexpr int kAhead = 4;  // heads that a thread has on their way at once

struct Token {
  int n, t, T;
  long nt;
};
__device__ __forceinline__ bool token_of(const KvArgs& a,
                                         const gdn::LaneTable& tl, int nt,
                                         Token& k) {
  if (nt >= a.lanes * a.t_max) return false;
  k.nt = nt;
  k.n = nt / a.t_max;
  k.t = nt - k.n * a.t_max;
  k.T = tl.v[k.n];
  return k.t < k.T;
}
// The token's page (-1: none) and its place in it; row h of the cache's heads
// is then that of (page h_kv + h) page_size + place.
__device__ __forceinline__ int page_for(const KvArgs& a, const Token& k,
                                        int& place) {
  place = 0;
  const int pos = slot_of(a, k.n, k.t, k.T);
  if (pos < 0) return -1;
  const int nth = page_of(a, pos);
  place = pos - nth * a.page;
  const int page = a.table[(long)k.n * a.max_pages + nth];
  return (unsigned)page < (unsigned)a.n_pages ? page : -1;
}

// Rows that are turned: queries, and keys unless they go into 4 bits.  A unit
// is eight pairs, or of neighbouring channels four.
template <typename T, bool FP4, bool PAIRS>
__device__ __forceinline__ void turn_rows(const RopeArgs& p,
                                          const gdn::LaneTable& tl, int d,
                                          const RopePlan& g, int i) {
  const KvArgs& a = p.kv;
  constexpr int kN = PAIRS ? 4 : 8, kParts = PAIRS ? 1 : 2;
  const int row = i / g.units, u = i - row * g.units;
  const int nt = row / g.slots, slot = row - nt * g.slots;
  Token k;
  if (!token_of(a, tl, nt, k)) return;
  const int queries = p.q ? a.h_q : 0;
  const int c0 = 8 * u, c1 = 8 * u + p.rot / 2;  // channels
  const T* q = (const T*)p.q + k.nt * p.qs;
  const T* kk = (const T*)p.k + k.nt * p.ks;
  auto source = [&](int h) {
    return h < queries ? q + (long)h * d : kk + (long)(h - queries) * d;
  };
  Turns<kN> w;
  w.set(turn_of(p, k.n, k.t, k.T), p.inv_freq + kN * u);
  int place, page = -1;
  if (!FP4) page = page_for(a, k, place);
#pragma unroll 1
  for (int h0 = slot; h0 < g.heads; h0 += kAhead * g.slots) {
    Eight x[kAhead], y[kAhead];
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int h = h0 + b * g.slots;
      const T* src = source(h < g.heads ? h : h0);
      x[b] = load_eight(src + c0);
      if (!PAIRS) y[b] = load_eight(src + c1);
    }
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      const int h = h0 + b * g.slots;
      if (h >= g.heads) break;
      T* dst;
      if (FP4 || h < queries) {
        dst = (T*)p.q_out + (k.nt * a.h_q + h) * d;
      } else {
        if (page < 0) break;  // (keys come last)
        dst = (T*)p.kc + (((long)page * a.h_kv + (h - queries)) * a.page + place) * d;
      }
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        float& l = x[b].x[PAIRS ? 2 * e : e];
        float& r = PAIRS ? x[b].x[(2 * e + 1) % 8] : y[b].x[e];
        const float a0 = l, b0 = r;
        l = a0 * w.c[e] - b0 * w.s[e];
        r = b0 * w.c[e] + a0 * w.s[e];
      }
      store_eight(dst + c0, x[b]);
      if (kParts == 2) store_eight(dst + c1, y[b]);
    }
  }
}

// Pieces that stay as they are: queries' and keys' channels from rot on, and
// values (keys and values unless they go into 4 bits).
template <typename T, bool FP4>
__device__ __forceinline__ void copy_rows(const RopeArgs& p,
                                          const gdn::LaneTable& tl, int d,
                                          const RopePlan& g, int i) {
  const KvArgs& a = p.kv;
  constexpr int kPer = 16 / sizeof(T);
  const int nt = i / g.pieces, at = i - nt * g.pieces;
  Token k;
  if (!token_of(a, tl, nt, k)) return;
  const int tail = (d - p.rot) / kPer, whole = d / kPer;
  const int of_q = p.q ? a.h_q * tail : 0, of_k = FP4 ? 0 : a.h_kv * tail;
  const T* src;
  T* dst;
  if (at < of_q) {
    const int h = at / tail, c = p.rot + (at - h * tail) * kPer;
    src = (const T*)p.q + k.nt * p.qs + (long)h * d + c;
    dst = (T*)p.q_out + (k.nt * a.h_q + h) * d + c;
  } else {
    const bool value = at >= of_q + of_k;
    const int j = value ? at - of_q - of_k : at - of_q;
    const int per = value ? whole : tail, h = j / per;
    const int c = (value ? 0 : p.rot) + (j - h * per) * kPer;
    int place;
    const int page = page_for(a, k, place);
    if (page < 0) return;
    src = (value ? (const T*)p.v + k.nt * p.vs : (const T*)p.k + k.nt * p.ks) +
          (long)h * d + c;
    dst = (T*)(value ? p.vc : p.kc) +
          (((long)page * a.h_kv + h) * a.page + place) * d + c;
  }
  *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
}

// Keys and values into 4 bits: eight neighbouring channels a thread, four
// threads a block of 32.  Keys are turned in f64: a code is half its value
// apart from the next, and of 10^7 keys off by steps of f32 a few would lie on
// the other side of the border between two.
template <typename T, bool PAIRS>
__device__ __forceinline__ void code_rows(const RopeArgs& p,
                                          const gdn::LaneTable& tl, int d,
                                          const RopePlan& g, int i) {
  const KvArgs& a = p.kv;
  const int units = d / 8, row = i / units, u = i - row * units;
  const int nt = row / g.slots4, slot = row - nt * g.slots4;
  Token k;
  if (!token_of(a, tl, nt, k)) return;
  const bool turns = 8 * u < p.rot;
  // channels 8 u .. are turned with those half of rot away
  const int hp = p.rot / 16;
  const bool second = !PAIRS && u >= hp;
  const int other = PAIRS || !turns ? u : second ? u - hp : u + hp;
  Turns<8, double> w;
  if (turns) {
    const int pos = turn_of(p, k.n, k.t, k.T);
    if constexpr (PAIRS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) turn(pos, p.inv_freq[4 * u + e], w.c[e], w.s[e]);
    } else {
      w.set(pos, p.inv_freq + 8 * (second ? other : u));
    }
  }
  int place;
  const int page = page_for(a, k, place);
  const T* ks = (const T*)p.k + k.nt * p.ks;
  const T* vs = (const T*)p.v + k.nt * p.vs;
  auto put = [&](const Fp4Rows& to, uint16_t* held, int h, const float (&x)[8]) {
    const Coded y = fp4_code(x);
    if (page >= 0) {
      const long at = ((long)page * a.h_kv + h) * a.page + place;
      *reinterpret_cast<uint32_t*>(to.codes + at * (d / 2) + 4 * u) = y.codes;
      if (u % 4 == 0) to.scales[at * (d / 32) + u / 4] = (uint8_t)y.scale;
    }
    if (held)
      *reinterpret_cast<u32x4*>(held + (k.nt * a.h_kv + h) * d + 8 * u) =
          fp4_values(y.codes, y.scale);
  };
  constexpr int kTwo = 2;  // heads on their way
#pragma unroll 1
  for (int h0 = slot; h0 < a.h_kv; h0 += kTwo * g.slots4) {
    Eight x[kTwo], y[kTwo], z[kTwo];
#pragma unroll
    for (int b = 0; b < kTwo; ++b) {
      const int h = h0 + b * g.slots4 < a.h_kv ? h0 + b * g.slots4 : h0;
      x[b] = load_eight(ks + (long)h * d + 8 * u);
      if (!PAIRS) y[b] = load_eight(ks + (long)h * d + 8 * other);
      z[b] = load_eight(vs + (long)h * d + 8 * u);
    }
#pragma unroll
    for (int b = 0; b < kTwo; ++b) {
      const int h = h0 + b * g.slots4;
      if (h >= a.h_kv) break;
      if (turns) {
        if constexpr (PAIRS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double l = x[b].x[2 * e], r = x[b].x[2 * e + 1];
            x[b].x[2 * e] = to_odd(l * w.c[e] - r * w.s[e]);
            x[b].x[2 * e + 1] = to_odd(r * w.c[e] + l * w.s[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[b].x[e] = to_odd((double)x[b].x[e] * w.c[e] +
                               (double)y[b].x[e] * (second ? w.s[e] : -w.s[e]));
        }
      }
      put(p.k4, p.k_held, h, x[b].x);
      put(p.v4, p.v_held, h, z[b].x);
    }
  }
}

template <typename T, bool FP4, bool PAIRS>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p,
                                                   gdn::LaneTable tl, int d,
                                                   RopePlan g) {
  int b = blockIdx.x;
  if (b < g.blocks)
    return turn_rows<T, FP4, PAIRS>(p, tl, d, g, b * 256 + threadIdx.x);
  b -= g.blocks;
  if (b < g.copy_blocks)
    return copy_rows<T, FP4>(p, tl, d, g, b * 256 + threadIdx.x);
  b -= g.copy_blocks;
  if constexpr (FP4) code_rows<T, PAIRS>(p, tl, d, g, b * 256 + threadIdx.x);
}

// ---------------------------------------------------------------- host side
static int check_rope(const char* fn, const gdn_kv_dims* dims,
                      const int32_t* t_lane, const void* q, int64_t q_stride,
                      const void* k, int64_t k_stride, const void* v,
                      int64_t v_stride, int dtype, const float* inv_freq,
                      int32_t rot_dim, const int32_t* positions,
                      const void* q_out, int flags, const int32_t* page_table,
                      const int32_t* kv_len, gdn::LaneTable& tl, int& any) {
  char msg[128];
  const auto bad = [&](int status, const char* what) {
    snprintf(msg, sizeof(msg), "%s: %s", fn, what);
    return fail(status, msg);
  };
  const int rc = check_kv_dims(fn, dims);
  if (rc != GDN_OK) return rc;
  const gdn_kv_dims& d = *dims;
  if (dtype != GDN_BF16 && dtype != GDN_F32) return bad(GDN_EINVAL, "unknown dtype");
  if (flags & ~GDN_FLAG_ROPE_PAIRS) return bad(GDN_EINVAL, "unknown flags");
  if (rot_dim < 0 || rot_dim > d.d || rot_dim % 16 != 0)
    return bad(GDN_EINVAL, "rot_dim must be a multiple of 16 in 0..d");
  if (!t_lane || !k || !v || !page_table || !kv_len || (q && !q_out) ||
      (!q && q_out) || (rot_dim > 0 && !inv_freq))
    return bad(GDN_EINVAL, "required pointer is NULL");
  const int per = dtype == GDN_BF16 ? 8 : 4;  // elements in 16 bytes
  const int64_t nq = (int64_t)d.h_q * d.d, nk = (int64_t)d.h_kv * d.d;
  const int64_t most = (int64_t)1 << 40;
  if ((q && (q_stride < nq || q_stride > most || q_stride % per != 0)) ||
      k_stride < nk || k_stride > most || k_stride % per != 0 ||
      v_stride < nk || v_stride > most || v_stride % per != 0)
    return bad(GDN_EINVAL, "a row stride is too small, too large or not a multiple of 16 bytes");
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) ||
      misaligned(q_out, 16) || misaligned(inv_freq, 4) ||
      misaligned(positions, 4) || misaligned(page_table, 4) ||
      misaligned(kv_len, 4))
    return bad(GDN_EINVAL, "misaligned pointer");
  return check_lanes(fn, d, t_lane, tl, any);
}

// Slots of heads for a token's `units` threads each: as many as bring the call
// to about kEnough threads (four rounds of 256 a CU), the fewest heads a thread:
// a small call has no work to spare for threads with many heads, a large one
// none for angles worked out again.
constexpr long kEnough = 256 * 1024;
static int slots_for(long tokens, int units, int heads) {
  const long n = (kEnough + tokens * units - 1) / (tokens * units);
  return n < heads ? (int)n : heads;
}

template <typename T, bool FP4>
static hipError_t run_rope(const RopeArgs& p, const gdn::LaneTable& tl, int d,
                           const RopePlan& g, dim3 grid, hipStream_t st) {
  return p.pairs
             ? launch(rope_kernel<T, FP4, true>, grid, dim3(256), st, p, tl, d, g)
             : launch(rope_kernel<T, FP4, false>, grid, dim3(256), st, p, tl, d, g);
}

static int launch_rope(const char* fn, const gdn_kv_dims& d, RopeArgs& p,
                       const gdn::LaneTable& tl, int dtype, bool fp4,
                       void* stream) {
  char msg[128];
  const int size = dtype == GDN_BF16 ? 2 : 4;
  const long tokens = (long)d.n_lanes * d.t_max;
  const int queries = p.q ? d.h_q : 0;
  RopePlan g;
  g.units = p.rot / (p.pairs ? 8 : 16);
  g.heads = queries + (fp4 ? 0 : d.h_kv);
  if (g.heads == 0) g.units = 0;
  g.slots = g.units > 0 ? slots_for(tokens, g.units, g.heads) : 1;
  const long pieces = ((queries + (fp4 ? 0l : d.h_kv)) * (d.d - p.rot) +
                       (fp4 ? 0l : (long)d.h_kv * d.d)) * size / 16;
  g.pieces = (int)pieces;
  g.slots4 = slots_for(tokens, d.d / 8, d.h_kv);
  const auto blocks = [](double n) { return (n + 255) / 256; };
  const double turning = blocks((double)tokens * g.slots * g.units);
  const double copying = blocks((double)tokens * pieces);
  const double coding = fp4 ? blocks((double)tokens * g.slots4 * (d.d / 8)) : 0;
  if ((turning + copying + coding) * 256 > (double)INT_MAX) {
    snprintf(msg, sizeof(msg), "%s: grid too large", fn);
    return fail(GDN_EINVAL, msg);
  }
  g.blocks = (int)turning;
  g.copy_blocks = (int)copying;
  const dim3 grid((unsigned)(g.blocks + g.copy_blocks + (int)coding));
  const hipStream_t st = (hipStream_t)stream;
  const hipError_t e =
      dtype == GDN_BF16
          ? fp4 ? run_rope<uint16_t, true>(p, tl, d.d, g, grid, st)
                : run_rope<uint16_t, false>(p, tl, d.d, g, grid, st)
          : fp4 ? run_rope<float, true>(p, tl, d.d, g, grid, st)
                : run_rope<float, false>(p, tl, d.d, g, grid, st);
  snprintf(msg, sizeof(msg), "%s launch", fn);
  return gdn::hip_status(e, msg);
}

}  // namespace gdnk

extern "C" int gdn_rope_append(
    const gdn_kv_dims* dims, const int32_t* t_lane, const void* q,
    int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, int dtype, const float* inv_freq, int32_t rot_dim,
    const int32_t* positions, void* q_out, void* k_cache, void* v_cache,
    const int32_t* page_table, const int32_t* kv_len, int flags,
    void* stream) {
  using namespace gdnk;
  const char* fn = "gdn_rope_append";
  gdn::LaneTable tl;
  int any;
  const int rc = check_rope(fn, dims, t_lane, q, q_stride, k, k_stride, v,
                            v_stride, dtype, inv_freq, rot_dim, positions,
                            q_out, flags, page_table, kv_len, tl, any);
  if (rc != GDN_OK) return rc;
  if (!k_cache || !v_cache)
    return fail(GDN_EINVAL, "gdn_rope_append: required pointer is NULL");
  if (misaligned(k_cache, 16) || misaligned(v_cache, 16))
    return fail(GDN_EINVAL, "gdn_rope_append: misaligned pointer");
  if (!any) return GDN_OK;
  RopeArgs p = {kv_args(*dims, k_cache, v_cache, page_table, kv_len),
                q, k, v, q_stride, k_stride, v_stride, q_out, k_cache, v_cache,
                {}, {}, nullptr, nullptr, inv_freq, positions, rot_dim,
                (flags & GDN_FLAG_ROPE_PAIRS) != 0};
  return launch_rope(fn, *dims, p, tl, dtype, false, stream);
}

extern "C" int gdn_rope_append_mxfp(
    const gdn_kv_dims* dims, const int32_t* t_lane, const void* q,
    int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, int dtype, const float* inv_freq, int32_t rot_dim,
    const int32_t* positions, void* q_out, uint8_t* k_codes,
    uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
    const int32_t* page_table, const int32_t* kv_len, void* k_held,
    void* v_held, int flags, void* stream) {
  using namespace gdnk;
  const char* fn = "gdn_rope_append_mxfp";
  gdn::LaneTable tl;
  int any;
  const int rc = check_rope(fn, dims, t_lane, q, q_stride, k, k_stride, v,
                            v_stride, dtype, inv_freq, rot_dim, positions,
                            q_out, flags, page_table, kv_len, tl, any);
  if (rc != GDN_OK) return rc;
  if (!k_codes || !k_scales || !v_codes || !v_scales)
    return fail(GDN_EINVAL, "gdn_rope_append_mxfp: required pointer is NULL");
  if (misaligned(k_codes, 16) || misaligned(k_scales, 16) ||
      misaligned(v_codes, 16) || misaligned(v_scales, 16) ||
      misaligned(k_held, 16) || misaligned(v_held, 16))
    return fail(GDN_EINVAL, "gdn_rope_append_mxfp: misaligned pointer");
  if (!rows_fit(*dims))
    return fail(GDN_EINVAL, "gdn_rope_append_mxfp: 2^32 rows or more in the cache");
  if (!any) return GDN_OK;
  RopeArgs p = {kv_args(*dims, nullptr, nullptr, page_table, kv_len),
                q, k, v, q_stride, k_stride, v_stride, q_out, nullptr, nullptr,
                {k_codes, k_scales}, {v_codes, v_scales},
                (uint16_t*)k_held, (uint16_t*)v_held, inv_freq, positions,
                rot_dim, (flags & GDN_FLAG_ROPE_PAIRS) != 0};
  return launch_rope(fn, *dims, p, tl, dtype, true, stream);
}
