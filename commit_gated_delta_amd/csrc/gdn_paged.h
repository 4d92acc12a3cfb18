// gdn_paged.h -- attention of draft windows or single tokens over a paged
// key-value cache, and the cache's writer (gdn_paged_attention,
// gdn_kv_append).  Compiled as part of gdn_state.hip.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_window_common.h"

namespace gdnk {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct KvArgs {
  const void *k, *v;  // the caches
  const int* table;
  const int* kv_len;
  int lanes, t_max, h_q, h_kv, page, n_pages, max_pages;
};

// Positions that lane n's cache holds.
__device__ __forceinline__ int lane_len(const KvArgs& a, int n) {
  const int cap = a.max_pages * a.page, len = a.kv_len[n];
  return len < 0 ? 0 : len > cap ? cap : len;
}

// First element of position pos's row of key-value head h, or -1 when its
// page is outside the cache.
__device__ __forceinline__ long row_of(const KvArgs& a, int n, int h, int pos,
                                       int d) {
  const int page = a.table[(long)n * a.max_pages + pos / a.page];
  if ((unsigned)page >= (unsigned)a.n_pages) return -1;
  return (((long)page * a.h_kv + h) * a.page + pos % a.page) * d;
}

__device__ __forceinline__ float elem(const uint16_t* p, long i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}
__device__ __forceinline__ float elem(const float* p, long i) { return p[i]; }

// One wave per (lane, token, query head): 64 positions at a time, a lane per
// position for the scores, a lane per D/64 columns for the values.
template <int D, typename T>
__global__ __launch_bounds__(64) void attend_kernel(KvArgs a,
                                                    gdn::LaneTable tl,
                                                    const T* __restrict__ q,
                                                    float* __restrict__ o,
                                                    float scale) {
  __shared__ float qs[D];
  __shared__ float ps[64];
  __shared__ long rows[64];
  const int lane = threadIdx.x;
  const int h = blockIdx.x % a.h_q, nt = blockIdx.x / a.h_q;
  const int n = nt / a.t_max, t = nt % a.t_max;
  const int T_n = tl.v[n];
  if (t >= T_n) return;
  const long qo = (long)blockIdx.x * D;
  const int hk = h / (a.h_q / a.h_kv);
  for (int i = lane; i < D; i += 64) qs[i] = elem(q, qo + i);
  __syncthreads();
  const int end = lane_len(a, n) - T_n + t + 1;
  float m = -INFINITY, l = 0.f, acc[D / 64] = {};
  for (int p0 = 0; p0 < end; p0 += 64) {
    const int pos = p0 + lane;
    const long row = pos < end ? row_of(a, n, hk, pos, D) : -1;
    float s = -INFINITY;
    if (row >= 0) {
      s = 0.f;
      for (int i = 0; i < D; ++i)
        s = __builtin_fmaf(qs[i], elem((const T*)a.k, row + i), s);
      s *= scale;
    }
    float tile = s;
    for (int x = 1; x < 64; x *= 2) tile = fmaxf(tile, __shfl_xor(tile, x));
    const float m2 = fmaxf(m, tile);
    const float keep = m == -INFINITY ? 0.f : expf(m - m2);
    const float e = row >= 0 ? expf(s - m2) : 0.f;
    l = l * keep + gdn::wave_sum(e);
    m = m2;
    __syncthreads();
    ps[lane] = e;
    rows[lane] = row;
    __syncthreads();
    for (int c = 0; c < D / 64; ++c) acc[c] *= keep;
    for (int j = 0; j < 64; ++j) {
      if (rows[j] < 0) continue;
      for (int c = 0; c < D / 64; ++c)
        acc[c] = __builtin_fmaf(ps[j],
                                elem((const T*)a.v, rows[j] + 64 * c + lane),
                                acc[c]);
    }
  }
  for (int c = 0; c < D / 64; ++c)
    o[qo + 64 * c + lane] = l > 0.f ? acc[c] / l : 0.f;
}

// One 16-byte piece of a key and of a value row per thread.
__global__ __launch_bounds__(256) void append_kernel(
    KvArgs a, gdn::LaneTable tl, const u32x4* __restrict__ k,
    const u32x4* __restrict__ v, u32x4* __restrict__ kc,
    u32x4* __restrict__ vc, int pieces) {
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  const long row = i / pieces;  // (lane, token, head)
  const int piece = (int)(i % pieces);
  const long nt = row / a.h_kv;
  const int h = (int)(row % a.h_kv);
  if (nt >= (long)a.lanes * a.t_max) return;
  const int n = (int)(nt / a.t_max), t = (int)(nt % a.t_max);
  const int T = tl.v[n];
  if (t >= T) return;
  const int pos = lane_len(a, n) - T + t;
  if (pos < 0) return;
  const long dst = row_of(a, n, h, pos, pieces);
  if (dst < 0) return;
  kc[dst + piece] = k[i];
  vc[dst + piece] = v[i];
}

// ---------------------------------------------------------------- host side
static int check_kv_dims(const char* fn, const gdn_kv_dims* p) {
  char msg[128];
  if (!p) {
    snprintf(msg, sizeof(msg), "%s: dims is NULL", fn);
    return fail(GDN_EINVAL, msg);
  }
  const gdn_kv_dims& d = *p;
  if (d.n_lanes < 1 || d.n_lanes > GDN_MAX_LANES || d.t_max < 1 ||
      d.t_max > GDN_MAX_T || d.h_kv < 1 || d.h_q < 1 || d.h_q % d.h_kv != 0 ||
      d.d < 1 || d.page_size < 1 || d.n_pages < 1 || d.max_pages < 1 ||
      (double)d.max_pages * d.page_size >= (double)(1 << 30) ||
      (double)d.n_lanes * d.t_max * d.h_q * 32 > (double)INT_MAX ||
      (double)d.n_pages * d.page_size * d.h_kv > 9.0e15) {
    snprintf(msg, sizeof(msg), "%s: dims out of range", fn);
    return fail(GDN_EINVAL, msg);
  }
  if (d.d != 64 && d.d != 128 && d.d != 256) {
    snprintf(msg, sizeof(msg), "%s: d must be 64, 128 or 256", fn);
    return fail(GDN_EUNSUPPORTED, msg);
  }
  return GDN_OK;
}

static int check_lanes(const char* fn, const gdn_kv_dims& d,
                       const int32_t* t_lane, gdn::LaneTable& tl, int& any) {
  memset(&tl, 0, sizeof(tl));
  any = 0;
  for (int n = 0; n < d.n_lanes; ++n) {
    if (t_lane[n] < 0 || t_lane[n] > d.t_max) {
      char msg[128];
      snprintf(msg, sizeof(msg), "%s: t_lane out of 0..t_max", fn);
      return fail(GDN_EINVAL, msg);
    }
    tl.v[n] = (uint8_t)t_lane[n];
    any |= t_lane[n];
  }
  return GDN_OK;
}

static KvArgs kv_args(const gdn_kv_dims& d, const void* k, const void* v,
                      const int32_t* table, const int32_t* kv_len) {
  return {k,     v,         table,   kv_len,    d.n_lanes, d.t_max,
          d.h_q, d.h_kv, d.page_size, d.n_pages, d.max_pages};
}

template <typename T>
static hipError_t attend(const gdn_kv_dims& d, const KvArgs& a,
                         const gdn::LaneTable& tl, const void* q, float* o,
                         float scale, hipStream_t st) {
  const dim3 grid((unsigned)((long)d.n_lanes * d.t_max * d.h_q));
  switch (d.d) {
    case 64:
      return launch(attend_kernel<64, T>, grid, dim3(64), st, a, tl,
                    (const T*)q, o, scale);
    case 128:
      return launch(attend_kernel<128, T>, grid, dim3(64), st, a, tl,
                    (const T*)q, o, scale);
    default:
      return launch(attend_kernel<256, T>, grid, dim3(64), st, a, tl,
                    (const T*)q, o, scale);
  }
}

}  // namespace gdnk

extern "C" size_t gdn_paged_attention_workspace_bytes(const gdn_kv_dims* dims) {
  if (gdnk::check_kv_dims("gdn_paged_attention_workspace_bytes", dims) !=
      GDN_OK)
    return 0;
  return 0;
}

extern "C" int gdn_paged_attention(const gdn_kv_dims* dims,
                                   const int32_t* t_lane, const void* q,
                                   const void* k_cache, const void* v_cache,
                                   int dtype, const int32_t* page_table,
                                   const int32_t* kv_len, float* o,
                                   void* workspace, size_t ws_bytes,
                                   float scale, void* stream) {
  using namespace gdnk;
  const char* fn = "gdn_paged_attention";
  int rc = check_kv_dims(fn, dims);
  if (rc != GDN_OK) return rc;
  if (!t_lane || !q || !k_cache || !v_cache || !page_table || !kv_len || !o)
    return fail(GDN_EINVAL, "gdn_paged_attention: required pointer is NULL");
  if (dtype != GDN_BF16 && dtype != GDN_F32)
    return fail(GDN_EINVAL, "gdn_paged_attention: unknown dtype");
  if (misaligned(q, 16) || misaligned(k_cache, 16) ||
      misaligned(v_cache, 16) || misaligned(o, 16) ||
      misaligned(workspace, 16) || misaligned(page_table, 4) ||
      misaligned(kv_len, 4))
    return fail(GDN_EINVAL, "gdn_paged_attention: misaligned pointer");
  const size_t need = gdn_paged_attention_workspace_bytes(dims);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_paged_attention: workspace too small");
  gdn::LaneTable tl;
  int any;
  rc = check_lanes(fn, *dims, t_lane, tl, any);
  if (rc != GDN_OK) return rc;
  if (!any) return GDN_OK;
  const KvArgs a = kv_args(*dims, k_cache, v_cache, page_table, kv_len);
  const hipError_t e =
      dtype == GDN_BF16
          ? attend<uint16_t>(*dims, a, tl, q, o, scale, (hipStream_t)stream)
          : attend<float>(*dims, a, tl, q, o, scale, (hipStream_t)stream);
  return gdn::hip_status(e, "gdn_paged_attention launch");
}

extern "C" int gdn_kv_append(const gdn_kv_dims* dims, const int32_t* t_lane,
                             const void* k, const void* v, int dtype,
                             void* k_cache, void* v_cache,
                             const int32_t* page_table, const int32_t* kv_len,
                             void* stream) {
  using namespace gdnk;
  const char* fn = "gdn_kv_append";
  int rc = check_kv_dims(fn, dims);
  if (rc != GDN_OK) return rc;
  if (!t_lane || !k || !v || !k_cache || !v_cache || !page_table || !kv_len)
    return fail(GDN_EINVAL, "gdn_kv_append: required pointer is NULL");
  if (dtype != GDN_BF16 && dtype != GDN_F32)
    return fail(GDN_EINVAL, "gdn_kv_append: unknown dtype");
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_cache, 16) ||
      misaligned(v_cache, 16) || misaligned(page_table, 4) ||
      misaligned(kv_len, 4))
    return fail(GDN_EINVAL, "gdn_kv_append: misaligned pointer");
  gdn::LaneTable tl;
  int any;
  rc = check_lanes(fn, *dims, t_lane, tl, any);
  if (rc != GDN_OK) return rc;
  if (!any) return GDN_OK;
  const KvArgs a = kv_args(*dims, k_cache, v_cache, page_table, kv_len);
  const int pieces = dims->d * (dtype == GDN_BF16 ? 2 : 4) / 16;
  const long n = (long)dims->n_lanes * dims->t_max * dims->h_kv * pieces;
  const long blocks = (n + 255) / 256;
  if (blocks > INT_MAX)
    return fail(GDN_EINVAL, "gdn_kv_append: grid too large");
  const hipError_t e =
      launch(append_kernel, dim3((unsigned)blocks), dim3(256),
             (hipStream_t)stream, a, tl, (const u32x4*)k, (const u32x4*)v,
             (u32x4*)k_cache, (u32x4*)v_cache, pieces);
  return gdn::hip_status(e, "gdn_kv_append launch");
}
