// gdn_rope.h -- the writer of the paged cache with the position rotation on
// the way (gdn_rope_append, gdn_rope_append_mxfp).  Compiled as part of
// gdn_state.hip.
//
// Channel pair (a, b) of a query or key row at position p turns by the angle
// p f_i (f_i the pair's inverse frequency):
//   a' = a cos - b sin,   b' = b cos + a sin.
// p f_i has at most 31 + 24 significant bits, so its product in f64 is exact
// to half a step, and it is reduced to a fraction of a turn there: the angle
// is as good at the far end of a long cache as at its start.
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

// cos and sin of p f.  The turn's fraction within [-1/8, 1/8] of the nearest
// quarter goes through the Taylor series of sine and cosine, whose next terms
// are below 2^-25 at pi / 4.
__device__ __forceinline__ void turn(int p, float f, float& c, float& s) {
  const double a = (double)p * (double)f;
  // 1 / (2 pi) in two parts
  constexpr double kHi = 0.15915494309189534561, kLo = -9.8393383375912e-18;
  const double whole = __builtin_rint(a * kHi);
  const double r =
      __builtin_fma(a, kHi, -whole) + a * kLo;  // -1/2 .. 1/2
  const double quarter = __builtin_rint(4.0 * r);
  const float x = (float)((r - 0.25 * quarter) * 6.28318530717958647693);
  const float y = x * x;
  float sn = __builtin_fmaf(y, 2.75573192e-6f, -1.98412698e-4f);
  sn = __builtin_fmaf(y, sn, 8.33333333e-3f);
  sn = __builtin_fmaf(y, sn, -1.66666667e-1f);
  sn = __builtin_fmaf(x * y, sn, x);
  float cs = __builtin_fmaf(y, -2.75573192e-7f, 2.48015873e-5f);
  cs = __builtin_fmaf(y, cs, -1.38888889e-3f);
  cs = __builtin_fmaf(y, cs, 4.16666667e-2f);
  cs = __builtin_fmaf(y, cs, -0.5f);
  cs = __builtin_fmaf(y, cs, 1.f);
  const int k = (int)quarter & 3;  // quarter turns
  const float u = k & 1 ? sn : cs, v = k & 1 ? cs : sn;
  c = k == 1 || k == 2 ? -u : u;
  s = k >= 2 ? -v : v;
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
template <typename T>
__device__ __forceinline__ void copy_eight(T* to, const T* from) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    reinterpret_cast<u32x4*>(to)[i] = reinterpret_cast<const u32x4*>(from)[i];
}

// Channels 8 u .. 8 u + 7 of a row after the rotation at position pos.
template <typename T>
__device__ __forceinline__ Eight turned(const RopeArgs& p, const T* row, int u,
                                        int pos) {
  Eight x = load_eight(row + 8 * u);
  if (8 * u >= p.rot) return x;
  if (p.pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float c, s;
      turn(pos, p.inv_freq[4 * u + i], c, s);
      const float a = x.x[2 * i], b = x.x[2 * i + 1];
      x.x[2 * i] = a * c - b * s;
      x.x[2 * i + 1] = b * c + a * s;
    }
    return x;
  }
  const int hp = p.rot / 16;  // pieces of half the rotated channels
  const bool second = u >= hp;
  const Eight y = load_eight(row + 8 * (second ? u - hp : u + hp));
  const float* f = p.inv_freq + 8 * (second ? u - hp : u);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float c, s;
    turn(pos, f[i], c, s);
    x.x[i] = x.x[i] * c + y.x[i] * (second ? s : -s);
  }
  return x;
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

// One thread per eight channels of a row of q, k or v.
template <typename T, bool FP4>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p,
                                                   gdn::LaneTable tl, int d) {
  const KvArgs& a = p.kv;
  const int units = d / 8, heads = (p.q ? a.h_q : 0) + 2 * a.h_kv;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(i % units);
  const long row = i / units, nt = row / heads;
  int h = (int)(row % heads);
  if (nt >= (long)a.lanes * a.t_max) return;
  const int n = (int)(nt / a.t_max), t = (int)(nt % a.t_max);
  const int T_n = tl.v[n];
  if (t >= T_n) return;
  const int pos = turn_of(p, n, t, T_n);
  if (p.q && h < a.h_q) {
    const T* src = (const T*)p.q + nt * p.qs + (long)h * d;
    T* dst = (T*)p.q_out + (nt * a.h_q + h) * d;
    // a thread turns both halves of its pairs, so that q_out may be q
    const int hp = p.pairs ? 0 : p.rot / 16;
    if (8 * u >= p.rot) {
      copy_eight(dst + 8 * u, src + 8 * u);
    } else if (p.pairs) {
      store_eight(dst + 8 * u, turned(p, src, u, pos));
    } else if (u < hp) {
      const Eight x = turned(p, src, u, pos), y = turned(p, src, u + hp, pos);
      store_eight(dst + 8 * u, x);
      store_eight(dst + 8 * (u + hp), y);
    }
    return;
  }
  if (p.q) h -= a.h_q;
  const bool value = h >= a.h_kv;
  if (value) h -= a.h_kv;
  const T* src = value ? (const T*)p.v + nt * p.vs + (long)h * d
                       : (const T*)p.k + nt * p.ks + (long)h * d;
  const int slot = slot_of(a, n, t, T_n);
  const long at = slot < 0 ? -1 : row_of(a, n, h, slot, 1);  // row of the cache
  if constexpr (FP4) {
    // (the four threads of a block of 32 channels are neighbours)
    const Eight x = value ? load_eight(src + 8 * u) : turned(p, src, u, pos);
    const Coded y = fp4_code(x.x);
    const Fp4Rows& to = value ? p.v4 : p.k4;
    if (at >= 0) {
      *reinterpret_cast<uint32_t*>(to.codes + at * (d / 2) + 4 * u) = y.codes;
      if (u % 4 == 0) to.scales[at * (d / 32) + u / 4] = y.scale;
    }
    uint16_t* held = value ? p.v_held : p.k_held;
    if (held)
      *reinterpret_cast<u32x4*>(held + (nt * a.h_kv + h) * d + 8 * u) =
          fp4_values(y.codes, y.scale);
  } else {
    if (at < 0) return;
    T* dst = (T*)(value ? p.vc : p.kc) + at * d + 8 * u;
    if (value || 8 * u >= p.rot) copy_eight(dst, src + 8 * u);
    else store_eight(dst, turned(p, src, u, pos));
  }
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

static int launch_rope(const char* fn, const gdn_kv_dims& d, RopeArgs& p,
                       const gdn::LaneTable& tl, int dtype, bool fp4,
                       void* stream) {
  char msg[128];
  const long rows =
      (long)d.n_lanes * d.t_max * ((p.q ? d.h_q : 0) + 2l * d.h_kv);
  const long blocks = (rows * (d.d / 8) + 255) / 256;
  if (blocks > INT_MAX) {
    snprintf(msg, sizeof(msg), "%s: grid too large", fn);
    return fail(GDN_EINVAL, msg);
  }
  const dim3 grid((unsigned)blocks), block(256);
  const hipStream_t st = (hipStream_t)stream;
  hipError_t e;
  if (dtype == GDN_BF16)
    e = fp4 ? launch(rope_kernel<uint16_t, true>, grid, block, st, p, tl, d.d)
            : launch(rope_kernel<uint16_t, false>, grid, block, st, p, tl, d.d);
  else
    e = fp4 ? launch(rope_kernel<float, true>, grid, block, st, p, tl, d.d)
            : launch(rope_kernel<float, false>, grid, block, st, p, tl, d.d);
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
