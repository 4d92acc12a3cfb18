// gdn_decay.h -- linear attention with a decay per head, in its recurrent
// form (gdn_decay_step) and over packed prompts (gdn_decay_prefill).
// Compiled as part of gdn_kda.hip (the library is a fixed set of translation
// units; the other sibling of the gated delta rule lives there).
//
//   S_t = a_t S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  a_t = exp(g_t)
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_mfma_op.h"
#include "gdn_window_common.h"

namespace gdnd {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;

using gdn::op::f32x4;
using gdn::op::Op;
using gdn::op::Special;
using gdn::op::u32x4;

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
// registers at DK = 128, loaded and stored as 128-byte row pieces (streamed:
// nothing reads a state again before every layer has run; 194 -> 179 us for
// windows of up to 16 on 8 lanes x 48 layers, then without a load ahead).  Its k and
// q entries are DK/8 consecutive ones of the token's row.  o needs one sum
// over the eight row groups per token.
// The next token's inputs are loaded while one is computed, with no branch
// before their use, from wave-uniform addresses (16 lanes x 48 heads of 64 x
// 32, windows of up to 33: 30 -> 20 us; one lane x 32 heads of 128 x 128,
// window of 64: 57 -> 42 us).
// A single token is bound by HBM (8 lanes x 32 heads, 34 MB: 8 us of which
// half is latency); a window by HBM and by its three f32 operations per state
// entry and token (8 lanes x 48 layers, up to 16 tokens: 0.87 GB in 172 us,
// 5.1 TB/s), and with few states by the latter's latency.
constexpr int kStepCols = 32;

// R consecutive entries of a row, as loaded.
template <typename TIn, int R>
struct RowRegs {
  static constexpr int kWords = R * (int)sizeof(TIn) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const TIn* __restrict__ p) {
    if constexpr (kWords == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kWords == 2) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x;
      w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 a = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = a[e];
      }
    }
  }
  __device__ __forceinline__ void expand(float (&x)[R]) const {
    if constexpr (sizeof(TIn) == 4) {
#pragma unroll
      for (int i = 0; i < R; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < R / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

// Four consecutive columns of a row, as loaded.  V4: their number is a
// multiple of four and the row 16-byte (bf16: 8-byte) aligned.  Columns past
// the last one read as others and are never stored, so that no load is behind
// a branch: at[e] is the column to read for e (V4: for e = 0).
template <typename TIn, bool V4>
struct ColRegs {
  uint32_t w[4];
  __device__ __forceinline__ void load(const TIn* __restrict__ row,
                                       const int (&at)[4]) {
    if constexpr (!V4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(TIn) == 4) w[e] = __float_as_uint(row[at[e]]);
        else w[e] = row[at[e]];
      }
    } else if constexpr (sizeof(TIn) == 4) {
      const u32x4 a = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(row + at[0]));
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = a[e];
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(row + at[0]);
      w[0] = a.x;
      w[1] = a.y;
    }
  }
  __device__ __forceinline__ f32x4 expand() const {
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if constexpr (sizeof(TIn) == 4) x[e] = __uint_as_float(w[e]);
      else if constexpr (!V4) x[e] = __uint_as_float(w[e] << 16);
      else
        x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    return x;
  }
};
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

// Sums over the eight row groups (lane bits 3, 4, 5) of four columns: lane
// halves and quarters trade places, so that each step adds half as many
// values and a lane ends up with column 2 * bit 4 + bit 5 of its four.
__device__ __forceinline__ float sum_groups(f32x4 y) {
  auto fold32 = [](float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(
        __float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const float a = fold32(y[0], y[1]), b = fold32(y[2], y[3]);
  const auto r = __builtin_amdgcn_permlane16_swap(
      __float_as_uint(a), __float_as_uint(b), false, false);
  const float x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  // rotate the 16 lanes by eight
  return x + __int_as_float(__builtin_amdgcn_update_dpp(
                 0, __float_as_int(x), 0x128, 0xf, 0xf, false));
}

// One head's chain over T tokens.  Pointers are at the first token's row of
// the head; qs, vs, gs are the token strides.  Without o, q is not used (but
// read: it may be k).
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
  int at[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    at[e] = V4 ? (c < dv ? c : col0) : (c + e < dv ? c + e : col0);
  // the inputs of the next token are on their way while one is computed
  RowRegs<TIn, R> kr, qr;
  ColRegs<TIn, V4> vr;
  float gr;
  auto fetch = [&](int t) {
    kr.load(k + t * qs + r0);
    qr.load(q + t * qs + r0);
    vr.load(v + t * vs, at);
    gr = g[t * gs];
  };
  fetch(0);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    ColRegs<float, V4> x;
    x.load(s_in + (long)(r0 + i) * dv, at);
    st[i] = x.expand();
  }
  for (int t = 0; t < T; ++t) {
    float kk[R], qq[R];
    kr.expand(kk);
    qr.expand(qq);
    const f32x4 vv = vr.expand();
    const float a = expf(gr);
    fetch(t + 1 < T ? t + 1 : t);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st[i][e] = __builtin_fmaf(kk[i], vv[e], a * st[i][e]);
    if (o) {
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __builtin_fmaf(qq[i], st[i][e], y[e]);
      const float x = sum_groups(y) * scale;
      const int col = col0 + 4 * (lane & 7) + 2 * (lane >> 4 & 1) + (lane >> 5);
      if (!(lane & 8) && col < dv) __builtin_nontemporal_store(x, o + t * vs + col);
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
  const long unit = (long)blockIdx.x * 4 + gdn::uniform(threadIdx.x / 64);
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
      (const TIn*)(p.o ? p.q : p.k) + qo, (const TIn*)p.k + qo, (const TIn*)p.v + vo,
      p.per_head ? p.g + (long)layer * p.h_v + h : p.g + tok * p.h_v + h,
      p.s_in + so, p.s_out ? p.s_out + so : nullptr, p.o ? p.o + vo : nullptr,
      ks, vs, p.per_head ? 0 : p.h_v, T, p.d_v, col0, p.scale);
}

// -------------------------------------------------------------- chunked form
// Prompts run in chunks of 64 tokens.  With b_t the sum of the chunk's gates
// up to token t, B the whole sum and S0 the state before the chunk:
//   o_t = scale (exp(b_t) S0^T q_t + sum_{s <= t} exp(b_t - b_s)(q_t.k_s) v_s)
//   S   = exp(B) S0 + sum_s k_s (exp(B - b_s) v_s)^T
// Four products per chunk: Q K^T, Q S0, P V and K^T W, all on the matrix
// cores.  bf16 operands enter exactly, f32 ones (S0, P, W) as three bf16
// parts whose sum is the f32 value itself (8 of its 24 bits each), so the
// products are those of f32.  (Two rounded parts left states and outputs
// 2.5e-6 off, against 1e-7.)  f32 inputs use the f32 matrix cores.
//
// The transposed forms are computed (O^T = S0^T Q^T + V^T P^T with
// P^T = mask(K Q^T)), because then every intermediate is born in the layout
// the next product reads, and only V and K need a transposed read from LDS:
//   * K Q^T leaves its 16 x 16 result at lane (g, n) as rows (tokens s)
//     4g + e of column (token t) n; two such tiles are the B operand of
//     V^T P^T when slot (g, e) of the 32-token step stands for token 4g + e
//     (e < 4) or 16 + 4g + e - 4 of it.
//   * the state is held as lane (g, n) = column n, rows 32 ks + 8 g + e: the
//     A operand of S0^T Q^T.  K^T W lands on it when row m of the A operand
//     stands for state row 8 (m / 4) + 4 a + m % 4 of its 32 (a = 0, 1 the
//     two halves).
//   * a token's decays belong to one lane (column n) of O^T.
// A workgroup of four waves takes 4 CW columns of d_v of one head; every
// wave holds its CW columns of the state in registers.  P is formed once per
// workgroup, its tiles shared out over the waves, and handed on through LDS
// as finished operands while the waves multiply the state.
//
// Long sequences are cut into segments so that a launch fills the GPU: a
// first pass forms each segment's own state (from zero) and decay, a scan
// turns those into the segments' start states, and the output pass runs all
// segments at once.
//
// Measured, 32,768 tokens x 32 heads of 128, bf16: states pass 126 us (540 MB,
// 4.3 TB/s), scan 14 us, output pass 301..317 us (1.39 GB, 4.5 TB/s).  Bound
// by the bytes, at nine tenths and more of a copy's 4.75 TB/s: 2.0 GB in all
// where 1.35 would do, since both passes read K and V from HBM.  (Matrix
// cores 41 % and vector ALUs 48 % busy in the output pass, two waves per SIMD
// being all that 250 registers leave.)
constexpr int kChunk = 64;

// Segments of the sequences: sequence s has the segments first[s] ..
// first[s + 1] - 1 of seg tokens each (the last one shorter).
struct SegTable {
  int n, seg;
  int cols;  // of d_v per workgroup
  int first[GDN_MAX_LANES + 1];
  int start[GDN_MAX_LANES + 1];  // token rows start[s] .. start[s + 1] - 1
};

struct ChunkArgs {
  DecayArgs a;
  int d_k;
  float* slots;  // [segments][h_v][d_k][d_v]: start states of the segments
  float* decay;  // [segments][h_v]: decay over a whole segment
};

// Sequence of a segment.
__device__ __forceinline__ int seq_of(const SegTable& t, int seg) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= seg) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Inclusive sum over the 64 lanes in f64 (DPP row shifts, then the sums of
// the rows before).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_part(double x) {
  const long v = __builtin_bit_cast(long, x);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
  const int hi =
      __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, ((long)hi << 32) | (uint32_t)lo);
}
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp_part<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8
  x += dpp_part<0x112, 0xf>(x);
  x += dpp_part<0x114, 0xf>(x);
  x += dpp_part<0x118, 0xf>(x);
  x += dpp_part<0x142, 0xa>(x);  // row_bcast 15 into rows 1 and 3
  x += dpp_part<0x143, 0xc>(x);  // row_bcast 31 into rows 2 and 3
  return x;
}

constexpr double kLog2e = 1.4426950408889634;

// Decays of a chunk's tokens, in LDS.  Sums of gates are kept in f64 and
// handed on as hi + lo pairs of f32 (in units of log 2), so that differences
// of large sums keep their small values.
struct Gates {
  float2 b[kChunk];      // sum of the gates up to the token
  float in[kChunk];      // exp(b_t)
  float out[kChunk];     // exp(B - b_t)
  float all;             // exp(B)
};

// The same of lane's token, before they go to LDS.
struct GateRegs {
  float hi, lo, in, out, all;
  // From the token's gate; the whole sum.
  __device__ __forceinline__ double make(float g) {
    g = g < -1000.f ? -1000.f : g;
    const double b = wave_scan((double)g * kLog2e);
    const long bits = __builtin_bit_cast(long, b);
    const double B = __builtin_bit_cast(
        double,
        ((long)__builtin_amdgcn_readlane((int)(bits >> 32), 63) << 32) |
            (uint32_t)__builtin_amdgcn_readlane((int)bits, 63));
    hi = (float)b;
    lo = (float)(b - (double)hi);
    in = __builtin_amdgcn_exp2f(hi);
    out = __builtin_amdgcn_exp2f((float)(B - b));
    all = __builtin_amdgcn_exp2f((float)B);
    return B;
  }
  __device__ __forceinline__ void store(Gates& G, int lane) const {
    G.b[lane] = make_float2(hi, lo);
    G.in[lane] = in;
    G.out[lane] = out;
    if (lane == 0) G.all = all;
  }
};

// 64 token rows of W entries of a tensor in transit from memory to LDS: each
// thread holds pieces of 16 bytes, kRows rows apart at one column.  The loads
// go through a buffer resource that ends with the last valid row, so that
// rows past it read as zero without a branch; columns past the row's n
// entries are sent out of range too.  VEC: rows are 16-byte aligned and n is
// a multiple of the piece; else entry by entry.
constexpr int kBufWord3 = 0x00020000;  // raw buffer resource
constexpr int kOutOfRange = 1 << 30;  // (64 rows are at most as long)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p,
                                                            int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes,
                                           kBufWord3);
}

template <typename TIn, int W, bool VEC, bool kColumns>
struct Transit {
  typedef gdn::op::Tile<TIn, W, kColumns> Tile;
  static constexpr int kPer = Tile::kPer;
  static constexpr int kRows = 256 * kPer / W;
  static constexpr int kPieces = kChunk / kRows;
  static_assert(!Tile::kSwizzled || kRows % 16 == 0,
                "the permutation repeats every 16 rows");
  u32x4 r[kPieces];
  int first, step, n;  // byte offset of the thread's first piece, row step

  __device__ __forceinline__ void init(long stride, int n_) {
    const int t = threadIdx.x / (W / kPer), c = threadIdx.x % (W / kPer) * kPer;
    n = n_;
    step = (int)(kRows * stride * (long)sizeof(TIn));
    first = c < n ? (int)((t * stride + c) * (long)sizeof(TIn)) : kOutOfRange;
  }
  // base: the chunk's first row; rows: its valid ones.  A resource per piece,
  // so that the pieces share one offset register.
  __device__ __forceinline__ void load(const TIn* base, long stride, int rows) {
    int bytes = (int)(((rows < kChunk ? rows : kChunk) - 1) * stride + n) *
                (int)sizeof(TIn);
    const char* at = (const char*)base;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const auto rs = buffer_of(at, bytes > 0 ? bytes : 0);
      at += step;
      bytes -= step;
      if constexpr (VEC) {
        r[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, first, 0, 0);
      } else {
        const int c = threadIdx.x % (W / kPer) * kPer;
        r[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int off = c + e < n ? first + e * (int)sizeof(TIn) : kOutOfRange;
          if constexpr (sizeof(TIn) == 4)
            r[i][e] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0);
          else
            r[i][e / 2] |= (uint32_t)(uint16_t)
                               __builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0)
                           << (16 * (e & 1));
        }
      }
    }
  }
  __device__ __forceinline__ void store(TIn* tile) const {
    const int t = threadIdx.x / (W / kPer), p = threadIdx.x % (W / kPer);
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      *reinterpret_cast<u32x4*>(tile + Tile::at(t, p) +
                                i * kRows * Tile::kPitch) = r[i];
  }
};

// What a chunk kernel is for: states alone (of all segments but the last of
// each sequence from zero, or with last_only of the last ones from their
// start states), or outputs and final states of all segments.
enum { kStates = 0, kOutput = 1 };

// Asks the scheduler to issue the region's matrix instructions one by one
// with V vector instructions after each, which run while it does.
template <int M, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
  }
}

// P^T in operand form: fragment (j, x) holds the token columns 16 j .. and
// the token rows 32 x .. 32 x + 31 (x <= j / 2), in this order; wave w makes
// the fragments kOwn[w] .. kOwn[w + 1] - 1.
constexpr int kFrags = 6;
constexpr int kFragJ[kFrags] = {0, 1, 2, 2, 3, 3};
constexpr int kFragX[kFrags] = {0, 0, 0, 1, 0, 1};
constexpr int kOwn[5] = {0, 2, 4, 5, 6};
__device__ constexpr int frag_of(int j, int x) { return j < 2 ? j : 2 * j - 2 + x; }

template <int DK, int CW, typename TIn, int MODE, bool VEC>
__global__ __launch_bounds__(256, sizeof(TIn) == 2 ? 2 : 1)
void chunk_kernel(ChunkArgs p, SegTable tab, int last_only) {
  typedef Op<TIn> O;
  typedef typename O::Raw Raw;
  typedef typename O::Wide Wide;
  constexpr int KS = DK / 32, CT = CW / 16, W = 4 * CW;
  typedef Transit<TIn, DK, true, MODE == kStates> KT;
  typedef Transit<TIn, W, VEC, true> VT;
  typedef typename KT::Tile KL;
  typedef typename VT::Tile VL;
  __shared__ __attribute__((aligned(16))) TIn Ks[kChunk * KL::kPitch];
  __shared__ __attribute__((aligned(16))) TIn Qs[MODE == kOutput ? kChunk * KL::kPitch : 8];
  __shared__ __attribute__((aligned(16))) TIn Vs[kChunk * VL::kPitch];
  __shared__ u32x4 Ps[MODE == kOutput ? kFrags : 1][O::kParts][64];
  __shared__ __attribute__((aligned(16))) Gates G;
  __shared__ int odd_chunk[2];  // whether a chunk's V holds special values

  const DecayArgs& a = p.a;
  const int ncb = (a.d_v + W - 1) / W;
  int item = gdn::xcd_item(blockIdx.x, gridDim.x);
  const int cb = item % ncb;
  item /= ncb;
  const int h = item % a.h_v;
  item /= a.h_v;
  int s, seg;
  if (last_only) {
    s = item;
    seg = tab.first[s + 1] - 1;
  } else if (MODE == kStates) {
    int lo = 0, hi = tab.n - 1;  // first[s] - s segments lie before sequence s
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (tab.first[mid] - mid <= item) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
    seg = item + s;
  } else {
    seg = item;
    s = seq_of(tab, seg);
  }
  const int nth = seg - tab.first[s], n_seg = tab.first[s + 1] - tab.first[s];
  const long tok0 = (long)tab.start[s] + (long)nth * tab.seg;
  const long rest = tab.start[s + 1] - tok0;
  const int T = rest < tab.seg ? (int)rest : tab.seg;
  const bool last = nth == n_seg - 1;

  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int hk = h / (a.h_v / a.h_k);
  const int col = cb * W, wcol = wave * CW;  // of d_v; of the block
  const int cols = a.d_v - col < W ? a.d_v - col : W;
  const long ks = (long)a.h_k * p.d_k, vs = (long)a.h_v * a.d_v;
  const TIn* K = (const TIn*)a.k + tok0 * ks + (long)hk * p.d_k;
  const TIn* Q = (const TIn*)a.q + tok0 * ks + (long)hk * p.d_k;
  const TIn* V = (const TIn*)a.v + tok0 * vs + (long)h * a.d_v + col;
  const float* __restrict__ g = a.per_head ? a.g + h : a.g + tok0 * a.h_v + h;
  const long gs = a.per_head ? 0 : a.h_v;
  float* out = MODE == kOutput ? a.o + tok0 * vs + (long)h * a.d_v + col : nullptr;

  // state entry (32 ks + 8 g4 + 4 a + e, column 16 ct + n): st[ct][ks][a][e]
  f32x4 st[CT][KS][2];
  const float* from = nullptr;
  if (MODE == kOutput || last_only) {
    if (n_seg > 1 && (nth > 0 || a.s_in))
      from = p.slots + ((long)seg * a.h_v + h) * p.d_k * a.d_v;
    else if (n_seg == 1 && a.s_in)
      from = a.s_in + ((long)s * a.h_v + h) * p.d_k * a.d_v;
  }
  // (rows past d_k lie behind the resource's end)
  const int state_bytes = (int)((long)p.d_k * a.d_v - col) * 4;
  const auto state_at = [&](int l, int ct, int i, int x, int e) {
    const int c = wcol + 16 * ct + (l & 15);
    return c < cols ? ((32 * i + 8 * (l >> 4) + 4 * x + e) * a.d_v + c) * 4
                    : kOutOfRange;
  };
  {
    const auto rs = buffer_of(from ? from + col : nullptr, from ? state_bytes : 0);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st[ct][i][x][e] =
                __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                    rs, state_at(lane, ct, i, x, e), 0, 0));
  }

  KT kt, qt;
  VT vt;
  kt.init(ks, p.d_k);
  qt.init(ks, p.d_k);
  vt.init(vs, cols);
  float gate = 0.f;
  double total = 0.0;
  GateRegs next_gates;
  auto fetch = [&](int t0) {
    const int rows = T - t0;
    kt.load(K + t0 * ks, ks, rows);
    vt.load(V + t0 * vs, vs, rows);
    gate = lane < rows ? g[(t0 + lane) * gs] : 0.f;
  };
  auto fetch_q = [&](int t0) {
    if constexpr (MODE == kOutput) qt.load(Q + t0 * ks, ks, T - t0);
  };
  auto place = [&](int left) {
    if constexpr (MODE == kOutput) {
      Special<TIn> odd;
#pragma unroll
      for (int i = 0; i < VT::kPieces; ++i) odd.look(vt.r[i]);
      if (odd.any()) odd_chunk[left & 1] = 1;
    }
    kt.store(Ks);
    if constexpr (MODE == kOutput) qt.store(Qs);
    vt.store(Vs);
    if (wave == 0) next_gates.store(G, lane);
  };

  // A segment's own state is summed from its last chunk to its first, each
  // chunk's writes decayed by the chunks summed before it: so the rows read
  // last, which the cache still holds, are those the output pass starts with.
  // (Such segments are whole chunks.)
  const bool back = MODE == kStates && !last_only;
  const int t_step = back ? -kChunk : kChunk;
  int t0 = back ? T - kChunk : 0;
  double sum = 0.0;  // of the chunk's gates
  if (T > 0) {
    fetch(t0);
    fetch_q(t0);
    sum = next_gates.make(gate);
  }
  int left = (T + kChunk - 1) / kChunk;  // chunks left
  if constexpr (MODE == kOutput) {
    if (tid == 0) odd_chunk[left & 1] = 0;
    __syncthreads();
  }
  if (T > 0) place(left);
  for (; left > 0; --left, t0 += t_step) {
    __syncthreads();
    if (MODE == kOutput && tid == 0) odd_chunk[~left & 1] = 0;
    const bool more = left > 1;
    const float since = back ? __builtin_amdgcn_exp2f((float)total) : 1.f;
    total += sum;
    // the next chunk's K and V rows now; Q's when the state's operands have
    // left the registers
    gate = 0.f;
    if (more) fetch(t0 + t_step);
    f32x4 acc[CT][4];
    const float all = back ? 1.f : G.all;
    if constexpr (MODE == kOutput) {
      // this wave's fragments of P^T
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (wave != w) continue;
#pragma unroll
        for (int f = kOwn[w]; f < kOwn[w + 1]; ++f) {
          const int j = kFragJ[f], x = kFragX[f], t = 16 * j + n;
          f32x4 pt[2];
          pt[0] = pt[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const Raw qf = O::template row<KL>(Qs, 16 * j, n, 4 * i + g4);
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (2 * x + y <= j)
                pt[y] = O::mul(
                    O::template row<KL>(Ks, 32 * x + 16 * y, n, 4 * i + g4),
                    qf, pt[y]);
          }
          const float2 bt = G.b[t];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if (2 * x + y > j) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int sr = 32 * x + 16 * y + 4 * g4 + e;
              const float2 bs = G.b[sr];
              const float w2 = __builtin_amdgcn_exp2f((bt.x - bs.x) +
                                                      (bt.y - bs.y));
              pt[y][e] = 2 * x + y < j || sr <= t ? pt[y][e] * w2 : 0.f;
            }
          }
          const Wide pw = O::wide(pt[0], pt[1]);
#pragma unroll
          for (int i = 0; i < O::kParts; ++i) Ps[f][i][lane] = pw.part[i];
        }
      }
      // O^T of the state: tokens 16 j + n, columns 16 ct + 4 g4 + e.  The
      // operands of a step of 32 state rows are made while the one before is
      // multiplied, and a state row is decayed as soon as it has been read.
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[ct][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      Wide sw[2][CT];
      constexpr int QB = sizeof(TIn) == 4 ? 2 : 1;  // (bf16: no registers left)
      Raw qf[QB][4];
      auto query_operands = [&](int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qf[i % QB][j] = O::template row<KL>(Qs, 16 * j, n, 4 * i + g4);
      };
      if constexpr (QB == 2) query_operands(0);
      auto state_operands = [&](int i) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          sw[i & 1][ct] = O::wide(st[ct][i][0], st[ct][i][1]);
          st[ct][i][0] *= all;
          st[ct][i][1] *= all;
        }
      };
      // (while it multiplies, a wave goes first on its SIMD: 318 -> 301 us for
      // 32,768 tokens x 32 heads)
      __builtin_amdgcn_s_setprio(1);
      state_operands(0);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (QB == 1) query_operands(i);
        else if (i + 1 < KS) query_operands(i + 1);
        if (i + 1 < KS) state_operands(i + 1);
#pragma unroll
        for (int m = 0; m < O::kSteps; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              acc[ct][j] =
                  O::step(m, sw[i & 1][ct], qf[i % QB][j], acc[ct][j]);
        interleave<12 * CT, 4>();
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float in = G.in[16 * j + n];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[ct][j] *= in;
      }
      __builtin_amdgcn_s_setprio(0);
      __syncthreads();  // P^T is complete
    } else {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x) st[ct][i][x] *= all;
    }
    if (more) fetch_q(t0 + kChunk);
    Raw vf[2][CT];
    auto value_operands = [&]() {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          vf[x][ct] =
              O::template column<VL>(Vs, 32 * x, wcol + 16 * ct, 4, lane);
    };
    if constexpr (MODE == kStates) value_operands();
    if constexpr (MODE == kOutput) {
      Wide pw[2];
      auto p_operand = [&](int f) {
#pragma unroll
        for (int i = 0; i < O::kParts; ++i) pw[f & 1].part[i] = Ps[f][i][lane];
      };
      if (!odd_chunk[left & 1]) {
        value_operands();
        p_operand(0);
#pragma unroll
        for (int f = 0; f < kFrags; ++f) {
          if (f + 1 < kFrags) p_operand(f + 1);
#pragma unroll
          for (int m = 0; m < O::kSteps; ++m)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              acc[ct][kFragJ[f]] = O::step(m, vf[kFragX[f]][ct], pw[f & 1],
                                           acc[ct][kFragJ[f]]);
        }
      } else {
        // an infinity or a NaN in V must not reach the tokens before its own
        // (the lane's number passes through an empty asm, or what follows
        // from it is kept in registers through the whole loop)
        int l = lane;
        asm volatile("" : "+v"(l));
        const int lc = wcol + 4 * (l >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll 1
          for (int sr = 0; sr < 16 * j + 16; ++sr) {
            if (sr > 16 * j + (l & 15)) continue;
            u32x4 part[O::kParts];
#pragma unroll
            for (int i = 0; i < O::kParts; ++i)
              part[i] = Ps[frag_of(j, sr >> 5)][i][4 * (sr & 12) + (l & 15)];
            const float pv = O::slot(part, 4 * (sr >> 4 & 1) + (sr & 3));
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int c = lc + 16 * ct + e;
                acc[ct][j][e] += pv * gdn::op::value_of(
                    Vs[VL::at(sr, c / VL::kPer) + c % VL::kPer]);
              }
          }
        }
        value_operands();
      }
      int bytes =
          (int)(((T - t0 < kChunk ? T - t0 : kChunk) - 1) * vs + cols) * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // rows past the last one fall behind the resource's end
        const auto rs = buffer_of(out + (t0 + 16 * j) * vs, bytes > 0 ? bytes : 0);
        bytes -= (int)(16 * vs * 4);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const int c = wcol + 16 * ct + 4 * g4;
          const int off = (int)(n * vs + c) * 4;
          const u32x4 y = __builtin_bit_cast(u32x4, acc[ct][j] * a.scale);
          if constexpr (VEC) {
            __builtin_amdgcn_raw_buffer_store_b128(
                y, rs, c < cols ? off : kOutOfRange, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __builtin_amdgcn_raw_buffer_store_b32(
                  y[e], rs, c + e < cols ? off + 4 * e : kOutOfRange, 0, 0);
          }
        }
      }
    }
    // the writes of the chunk's tokens
    Wide ww[2][CT];
    Raw kf[2][2];
    auto write_operands = [&](int x) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(&G.out[32 * x + 4 * g4]);
      const f32x4 w1 =
          *reinterpret_cast<const f32x4*>(&G.out[32 * x + 16 + 4 * g4]);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        ww[x][ct] = MODE == kStates ? O::scaled(vf[x][ct], w0 * since, w1 * since)
                                    : O::scaled(vf[x][ct], w0, w1);
    };
    auto key_operands = [&](int u) {  // u = 32-token step x, 32 state rows i
#pragma unroll
      for (int y = 0; y < 2; ++y)
        kf[u & 1][y] = O::template column<KL>(Ks, 32 * (u / KS),
                                              32 * (u % KS) + 4 * y, 8, lane);
    };
    __builtin_amdgcn_s_setprio(1);
    key_operands(0);
    write_operands(0);
#pragma unroll
    for (int u = 0; u < 2 * KS; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      if (u + 1 < 2 * KS) key_operands(u + 1);
      if (u == KS - 1) write_operands(1);
      if (u == KS) sum = next_gates.make(gate);
#pragma unroll
      for (int m = 0; m < O::kSteps; ++m)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
            st[ct][u % KS][y] = O::step(m, kf[u & 1][y], ww[u / KS][ct],
                                        st[ct][u % KS][y]);
      if (u == KS - 1 || u == KS) interleave<6 * CT, 10>();
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    __syncthreads();
    if (more) place(left - 1);
  }

  float* to = nullptr;
  if (MODE == kStates && !last_only) {
    to = p.slots + ((long)(seg + 1) * a.h_v + h) * p.d_k * a.d_v;
    if (tid == 0 && cb == 0)
      p.decay[(long)seg * a.h_v + h] = __builtin_amdgcn_exp2f((float)total);
  } else if (last && a.s_out) {
    to = a.s_out + ((long)s * a.h_v + h) * p.d_k * a.d_v;
  }
  if (to) {
    // the offsets are computed anew: kept from the load at the kernel's start
    // they would cost 64 registers through the whole loop
    int l = lane;
    asm volatile("" : "+v"(l));
    const auto rs = buffer_of(to + col, state_bytes);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            __builtin_amdgcn_raw_buffer_store_b32(
                __float_as_uint(st[ct][i][x][e]), rs,
                state_at(l, ct, i, x, e), 0, 0);
  }
}

// Start states of the segments of every sequence that has more than one:
// slot 0 becomes S_init, slot i + 1 (which holds segment i's own state)
// decay_i * start_i + own_i.  One thread per state entry, the own states of
// eight segments in flight at a time.
__global__ __launch_bounds__(256) void segment_scan_kernel(ChunkArgs p,
                                                           SegTable tab) {
  const DecayArgs& a = p.a;
  const long size = (long)p.d_k * a.d_v;
  const long per_head = (size + 255) / 256;
  const long blk = blockIdx.x;
  const long at = blk % per_head * 256 + threadIdx.x;
  const int h = (int)(blk / per_head % a.h_v);
  const int s = (int)(blk / per_head / a.h_v);
  const int first = tab.first[s], n_seg = tab.first[s + 1] - first;
  if (n_seg < 2 || at >= size) return;
  float* slot = p.slots + ((long)first * a.h_v + h) * size + at;
  const float* dec = p.decay + (long)first * a.h_v + h;
  const long step = a.h_v * size;
  float S = 0.f;
  if (a.s_in) {
    S = a.s_in[((long)s * a.h_v + h) * size + at];
    slot[0] = S;
  }
  constexpr int kAhead = 8;
  for (int i = 0; i < n_seg - 1; i += kAhead) {
    float own[kAhead], d[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u < n_seg - 1) {
        own[u] = slot[(i + u + 1) * step];
        d[u] = dec[(long)(i + u) * a.h_v];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i + u < n_seg - 1) {
        S = __builtin_fmaf(d[u], S, own[u]);
        slot[(i + u + 1) * step] = S;
      }
  }
}

// ---------------------------------------------------------------- host side
static int check_heads(const char* fn, int h_v, int h_k, int d_k, int d_v) {
  char msg[128];
  // (64 token rows of a tensor are addressed with 31 bits)
  if (h_v < 1 || h_k < 1 || h_v % h_k != 0 || d_k < 1 || d_v < 1 ||
      d_v > 1024 || (double)h_v * d_v * 4 * 64 > (double)INT_MAX / 2 ||
      (double)h_k * d_k * 4 * 64 > (double)INT_MAX / 2) {
    snprintf(msg, sizeof(msg), "%s: sizes out of range", fn);
    return fail(GDN_EINVAL, msg);
  }
  if (d_k != 16 && d_k != 32 && d_k != 64 && d_k != 128) {
    snprintf(msg, sizeof(msg), "%s: d_k must be 16, 32, 64 or 128", fn);
    return fail(GDN_EUNSUPPORTED, msg);
  }
  return GDN_OK;
}

// (a call without tokens reads no inputs)
static int check_pointers(const char* fn, const DecayArgs& p, int in_dtype,
                          bool tokens) {
  char msg[128];
  const char* what = nullptr;
  if (tokens && (!p.k || !p.v || !p.g || (p.o && !p.q))) what = "required pointer is NULL";
  else if (in_dtype != GDN_BF16 && in_dtype != GDN_F32) what = "unknown in_dtype";
  else if (misaligned(p.q, 16) || misaligned(p.k, 16) || misaligned(p.v, 16) ||
           misaligned(p.g, 4) || misaligned(p.s_in, 16) ||
           misaligned(p.s_out, 16) || misaligned(p.o, 16))
    what = "pointers must be 16-byte aligned (g: 4-byte)";
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

// Sequences and segments of a prefill call.  Segments are as long as it
// takes for about two workgroups per CU (one launch then fills the GPU at the
// kernel's occupancy), and at least kMinSeg tokens: a segment costs its state
// twice written and twice read and its keys and values read once more.
// Measured for 7 f32 sequences of up to 1000 tokens on 8 heads: 68, 41, 27 us
// with segments of at least 512, 256 and 128 tokens.  A call whose sequences
// all have at most four chunks is not worth the two more launches.
// Workgroups take 128 columns of d_v, or 64 where that is all there are or
// where wider ones would not even be one per CU (kNarrowBlocks): with 64 a
// chunk takes less time, if more in all.  1024 tokens x 16 heads 34 -> 28 us,
// 200 x 32 heads 27 -> 19 us, 250 x 8 f32 heads 57 -> 36 us; with up to two a
// CU 131,072 x 4 heads would take 289 against 250 us.
constexpr int kTargetBlocks = 512;
constexpr int kMinSeg = 2 * kChunk;
constexpr int kWhole = 4 * kChunk;
constexpr int kNarrowBlocks = 256;

// The number of tokens, or -1 for bad lengths.
static long plan_segments(int32_t n_seqs, const int32_t* seq_len, int h_v,
                          int d_v, SegTable& t) {
  if (n_seqs < 1 || n_seqs > GDN_MAX_LANES || !seq_len) return -1;
  memset(&t, 0, sizeof(t));
  t.n = n_seqs;
  long tokens = 0, chunks = 0, longest = 0;
  for (int i = 0; i < n_seqs; ++i) {
    if (seq_len[i] < 0) return -1;
    tokens += seq_len[i];
    if (tokens > INT_MAX) return -1;
    chunks += (seq_len[i] + (long)kChunk - 1) / kChunk;
    if (seq_len[i] > longest) longest = seq_len[i];
    t.start[i + 1] = (int)tokens;
  }
  t.cols = d_v <= 64 ? 64 : 128;
  const long work = chunks * h_v * ((d_v + t.cols - 1) / t.cols);
  long seg = (work + kTargetBlocks - 1) / kTargetBlocks * kChunk;
  if (seg < kMinSeg) seg = kMinSeg;
  if (longest <= kWhole) seg = kWhole;
  if (seg > (1 << 30)) seg = 1 << 30;
  t.seg = (int)seg;
  for (int i = 0; i < n_seqs; ++i) {
    const long n = (seq_len[i] + seg - 1) / seg;
    t.first[i + 1] = t.first[i] + (int)(n < 1 ? 1 : n);
  }
  // with less than a workgroup per CU, narrower ones are done sooner
  if ((long)t.first[n_seqs] * h_v * ((d_v + t.cols - 1) / t.cols) <= kNarrowBlocks)
    t.cols = 64;
  return tokens;
}

// Workspace: a slot per segment and head, then the segments' decays.  Slots
// of sequences of one segment stay unused.
static size_t slots_bytes(const SegTable& t, int h_v, int d_k, int d_v) {
  return (size_t)t.first[t.n] * h_v * d_k * d_v * sizeof(float);
}
static size_t workspace_bytes(const SegTable& t, int h_v, int d_k, int d_v) {
  if (t.first[t.n] == t.n) return 0;
  return (slots_bytes(t, h_v, d_k, d_v) + 255) / 256 * 256 +
         (size_t)t.first[t.n] * h_v * sizeof(float);
}

template <int MODE, typename... Args>
static hipError_t launch_chunks(int d_k, int d_v, int w, int in_dtype, bool vec,
                                long items, hipStream_t st, Args&&... args) {
  const dim3 grid((unsigned)(items * ((d_v + w - 1) / w)));
  auto go = [&](auto dk, auto cw, auto t, auto v) {
    return launch(chunk_kernel<decltype(dk)::value, decltype(cw)::value,
                               decltype(t), MODE, decltype(v)::value>,
                  grid, dim3(256), st, args...);
  };
  auto of_vec = [&](auto dk, auto cw, auto t) {
    if (vec) return go(dk, cw, t, std::true_type{});
    return go(dk, cw, t, std::false_type{});
  };
  auto of_type = [&](auto dk, auto cw) {
    if (in_dtype == GDN_BF16) return of_vec(dk, cw, uint16_t{});
    return of_vec(dk, cw, float{});
  };
  auto of_cols = [&](auto dk) {
    if (w == 64) return of_type(dk, std::integral_constant<int, 16>{});
    return of_type(dk, std::integral_constant<int, 32>{});
  };
  if (d_k <= 32) return of_cols(std::integral_constant<int, 32>{});
  if (d_k == 64) return of_cols(std::integral_constant<int, 64>{});
  return of_cols(std::integral_constant<int, 128>{});
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
  rc = check_pointers(fn, p, in_dtype, true);
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
  SegTable t;
  if (check_heads("gdn_decay_prefill_workspace_bytes", h_v, h_k, d_k, d_v) !=
          GDN_OK ||
      plan_segments(n_seqs, seq_len, h_v, d_v, t) < 0)
    return 0;
  return workspace_bytes(t, h_v, d_k, d_v);
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
  SegTable tab;
  const long tokens = plan_segments(n_seqs, seq_len, h_v, d_v, tab);
  if (tokens < 0)
    return fail(GDN_EINVAL, "gdn_decay_prefill: bad n_seqs or seq_len");
  if (flags & ~GDN_FLAG_HEAD_DECAY)
    return fail(GDN_EINVAL, "gdn_decay_prefill: unknown flag bits");
  if (!o && !S_final)
    return fail(GDN_EINVAL,
                "gdn_decay_prefill: neither states nor outputs are wanted");
  ChunkArgs p = {{q, k, v, g, S_init, S_final, o, scale, 1, n_seqs, h_v, h_k,
                  d_v, 0, (flags & GDN_FLAG_HEAD_DECAY) ? 1 : 0},
                 d_k, nullptr, nullptr};
  rc = check_pointers(fn, p.a, in_dtype, tokens > 0);
  if (rc != GDN_OK) return rc;
  const size_t need = workspace_bytes(tab, h_v, d_k, d_v);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_decay_prefill: workspace too small");
  if (need > 0 && misaligned(workspace, 16))
    return fail(GDN_EINVAL,
                "gdn_decay_prefill: pointers must be 16-byte aligned");
  if (tokens == 0 && !S_final) return GDN_OK;
  const int w = tab.cols, segs = tab.first[n_seqs];
  const double scan = ((double)d_k * d_v + 255) / 256;
  if ((double)segs * h_v * ((d_v + w - 1) / w) > (double)INT_MAX ||
      (double)n_seqs * h_v * scan > (double)INT_MAX)
    return fail(GDN_EINVAL, "gdn_decay_prefill: grid too large");
  hipStream_t st = (hipStream_t)stream;
  const bool vec = d_v % (in_dtype == GDN_BF16 ? 8 : 4) == 0;
  hipError_t e = hipSuccess;
  if (segs > n_seqs) {
    p.slots = (float*)workspace;
    p.decay = (float*)((char*)workspace +
                       (slots_bytes(tab, h_v, d_k, d_v) + 255) / 256 * 256);
    e = launch_chunks<kStates>(d_k, d_v, w, in_dtype, vec,
                              (long)(segs - n_seqs) * h_v, st, p, tab, 0);
    if (e == hipSuccess)
      e = launch(segment_scan_kernel,
                 dim3((unsigned)((((long)d_k * d_v + 255) / 256) * h_v *
                                 n_seqs)),
                 dim3(256), st, p, tab);
  }
  // without outputs only the last segments are left to run
  if (e == hipSuccess && o)
    e = launch_chunks<kOutput>(d_k, d_v, w, in_dtype, vec, (long)segs * h_v, st,
                               p, tab, 0);
  else if (e == hipSuccess)
    e = launch_chunks<kStates>(d_k, d_v, w, in_dtype, vec, (long)n_seqs * h_v, st,
                               p, tab, 1);
  return gdn::hip_status(e, "gdn_decay_prefill launch");
}
