// gdn_paged_mxfp.h -- attention of draft windows or single tokens over a paged
// key-value cache held in 4 bits (gdn_paged_attention_mxfp).  Compiled as part
// of gdn_state.hip.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_mxfp.h"
#include "gdn_paged.h"

namespace gdnk {

struct Attend4Args {
  KvArgs kv;
  Fp4Rows k4, v4;
  const void* q;
  float* o;
  float scale;
};

// One workgroup per row of q: 256 positions at a time, a thread a position
// for the scores and a thread a channel for the values.
template <typename T>
__global__ __launch_bounds__(256) void attend4_kernel(Attend4Args p,
                                                      gdn::LaneTable tl, int d) {
  __shared__ float qs[256], ps[256];
  __shared__ long at[256];
  __shared__ float red[2][4];
  const KvArgs& a = p.kv;
  const int h = blockIdx.x % a.h_q;
  const long nt = blockIdx.x / a.h_q;
  const int n = (int)(nt / a.t_max), t = (int)(nt % a.t_max);
  const int T_n = tl.v[n];
  if (t >= T_n) return;
  const int hk = h / (a.h_q / a.h_kv), len = lane_len(a, n);
  const int end = len - T_n + t + 1;  // positions seen
  const int tid = threadIdx.x;
  const long row = (nt * a.h_q + h) * d;
  qs[tid] = tid < d ? elem((const T*)p.q, row + tid) : 0.f;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  bool any = false;
  __syncthreads();
  for (int p0 = 0; p0 < end; p0 += 256) {
    const int pos = p0 + tid;
    long r = -1;
    float x = -INFINITY;
    if (pos < end) r = row_of(a, n, hk, pos, 1);
    if (r >= 0) {
      x = 0.f;
      for (int c = 0; c < d; c += 8) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p.k4.codes + r * (d / 2) + c / 2);
        const codes_u32x4 v = fp4_values(w, p.k4.scales[r * (d / 32) + c / 32]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x += qs[c + 2 * i] * __uint_as_float(v[i] << 16);
          x += qs[c + 2 * i + 1] * __uint_as_float(v[i] & 0xffff0000u);
        }
      }
      x *= p.scale;
    }
    float top = x, sum = r >= 0 ? 1.f : 0.f;
    for (int i = 1; i < 64; i *= 2) {
      const float o = __shfl_xor(top, i);
      top = top != top || o != o ? NAN : fmaxf(top, o);
      sum += __shfl_xor(sum, i);
    }
    if (tid % 64 == 0) {
      red[0][tid / 64] = top;
      red[1][tid / 64] = sum;
    }
    at[tid] = r;
    __syncthreads();
    for (int w = 0; w < 4; ++w) {
      any |= red[1][w] > 0.f;
      const float o = red[0][w];
      top = top != top || o != o ? NAN : fmaxf(top, o);
    }
    const float next = top != top || m != m ? NAN : fmaxf(m, top);
    const float keep = next == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - next);
    const float e = r < 0 || next == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x - next);
    ps[tid] = e;
    m = next;
    __syncthreads();
    acc *= keep;
    l *= keep;
    const int stop = end - p0 < 256 ? end - p0 : 256;
    for (int i = 0; i < stop; ++i) {
      l += ps[i];
      if (tid < d && at[i] >= 0) {
        const uint32_t w = p.v4.codes[at[i] * (d / 2) + tid / 2];
        const uint32_t v = fp4_values(w, p.v4.scales[at[i] * (d / 32) + tid / 32])[0];
        acc += ps[i] * __uint_as_float(tid & 1 ? v & 0xffff0000u : v << 16);
      }
    }
    __syncthreads();
  }
  if (tid < d)
    p.o[row + tid] = !any ? 0.f : m == -INFINITY ? NAN : acc / l;
}

}  // namespace gdnk

extern "C" size_t gdn_paged_attention_mxfp_workspace_bytes(
    const gdn_kv_dims* dims) {
  if (gdnk::check_kv_dims("gdn_paged_attention_mxfp_workspace_bytes", dims) !=
      GDN_OK)
    return 0;
  return gdnk::attend_bytes(*dims);
}

extern "C" int gdn_paged_attention_mxfp(
    const gdn_kv_dims* dims, const int32_t* t_lane, const void* q, int dtype,
    const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
    const uint8_t* v_scales, const int32_t* page_table, const int32_t* kv_len,
    float* o, void* workspace, size_t ws_bytes, float scale, void* stream) {
  using namespace gdnk;
  const char* fn = "gdn_paged_attention_mxfp";
  int rc = check_kv_dims(fn, dims);
  if (rc != GDN_OK) return rc;
  if (!t_lane || !q || !k_codes || !k_scales || !v_codes || !v_scales ||
      !page_table || !kv_len || !o)
    return fail(GDN_EINVAL, "gdn_paged_attention_mxfp: required pointer is NULL");
  if (dtype != GDN_BF16 && dtype != GDN_F32)
    return fail(GDN_EINVAL, "gdn_paged_attention_mxfp: unknown dtype");
  if (misaligned(q, 16) || misaligned(k_codes, 16) || misaligned(k_scales, 16) ||
      misaligned(v_codes, 16) || misaligned(v_scales, 16) || misaligned(o, 16) ||
      misaligned(workspace, 16) || misaligned(page_table, 4) ||
      misaligned(kv_len, 4))
    return fail(GDN_EINVAL, "gdn_paged_attention_mxfp: misaligned pointer");
  const size_t need = gdn_paged_attention_mxfp_workspace_bytes(dims);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_paged_attention_mxfp: workspace too small");
  gdn::LaneTable tl;
  int any;
  rc = check_lanes(fn, *dims, t_lane, tl, any);
  if (rc != GDN_OK) return rc;
  if (!any) return GDN_OK;
  Attend4Args p = {kv_args(*dims, nullptr, nullptr, page_table, kv_len),
                   {(uint8_t*)k_codes, (uint8_t*)k_scales},
                   {(uint8_t*)v_codes, (uint8_t*)v_scales},
                   q, o, scale * kLog2e};
  const dim3 grid((unsigned)((long)dims->n_lanes * dims->t_max * dims->h_q));
  const hipError_t e =
      dtype == GDN_BF16
          ? launch(attend4_kernel<uint16_t>, grid, dim3(256), (hipStream_t)stream, p, tl, dims->d)
          : launch(attend4_kernel<float>, grid, dim3(256), (hipStream_t)stream, p, tl, dims->d);
  return gdn::hip_status(e, "gdn_paged_attention_mxfp launch");
}
