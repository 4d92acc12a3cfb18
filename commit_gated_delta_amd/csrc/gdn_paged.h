// gdn_paged.h -- attention of draft windows or single tokens over a paged
// key-value cache, and the cache's writer (gdn_paged_attention,
// gdn_kv_append).  Compiled as part of gdn_state.hip.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_mfma_op.h"
#include "gdn_window_common.h"

namespace gdnk {

using gdn::fail;
using gdn::launch;
using gdn::misaligned;

using gdn::op::f32x4;
using gdn::op::Op;
using gdn::op::Special;
using gdn::op::Tile;
using gdn::op::u32x4;

struct KvArgs {
  const void *k, *v;  // the caches
  const int* table;
  const int* kv_len;
  int lanes, t_max, h_q, h_kv, page, n_pages, max_pages;
  uint32_t page_mul;  // pos / page = (umulhi(pos, page_mul) + pos) >> page_shift
  int page_shift;
};

// Positions that lane n's cache holds.
__device__ __forceinline__ int lane_len(const KvArgs& a, int n) {
  const int cap = a.max_pages * a.page, len = a.kv_len[n];
  return len < 0 ? 0 : len > cap ? cap : len;
}

// First element of position pos's row of key-value head h, or -1 when its
// page is outside the cache.
__device__ __forceinline__ int page_of(const KvArgs& a, int pos) {
  return (int)((__umulhi((uint32_t)pos, a.page_mul) + (uint32_t)pos) >>
               a.page_shift);
}
__device__ __forceinline__ long row_in(const KvArgs& a, int page, int h,
                                       int row, int d) {
  if ((unsigned)page >= (unsigned)a.n_pages) return -1;
  return (((long)page * a.h_kv + h) * a.page + row) * d;
}
__device__ __forceinline__ long row_of(const KvArgs& a, int n, int h, int pos,
                                       int d) {
  const int nth = page_of(a, pos);
  return row_in(a, a.table[(long)n * a.max_pages + nth], h, pos - nth * a.page,
                d);
}

// --------------------------------------------------------- splitting the work
// A lane's positions are taken in units of kUnit, and the units of all lanes
// are shared out in splits of equally many, about `target` of them, whatever
// the lengths (which only the device knows).  Splits are numbered lane by
// lane; the grid holds the most there can be, target + lanes (each lane's
// last split may be a short one), and those past the last one end at once.
// Partial results of lanes with more than one split have a slot each, at most
// 2 * target of them.
constexpr int kUnit = 128;

struct Split {
  int lane;    // -1: no such split
  int len;     // positions of the lane
  int nth, n;  // this split among the lane's
  int units;   // units per split
  int slot;    // slot of the lane's first split
};

__device__ __forceinline__ int wave_scan_int(int x) {  // inclusive
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// The split `item`, or with of_lane the first split of lane `item`.  Every
// wave works it out for itself, 64 lanes at a time.
__device__ __forceinline__ Split find_split(const KvArgs& a,
                                            const gdn::LaneTable& tl, int item,
                                            int target, bool of_lane) {
  const int l = threadIdx.x & 63;
  int len[GDN_MAX_LANES / 64], u[GDN_MAX_LANES / 64], all = 0;
#pragma unroll
  for (int c = 0; c < GDN_MAX_LANES / 64; ++c) {
    const int n = 64 * c + l;
    const bool on = n < a.lanes && tl.v[n < a.lanes ? n : 0] > 0;
    len[c] = on ? lane_len(a, n) : 0;
    u[c] = (len[c] + kUnit - 1) / kUnit;
    if (on && u[c] == 0) u[c] = 1;  // its outputs are zeros
    all += u[c];
  }
  all = __builtin_amdgcn_readlane(wave_scan_int(all), 63);
  Split s;
  s.units = (all + target - 1) / target;
  if (s.units < 1) s.units = 1;
  // (no lane has more, and so many positions still fit an int)
  constexpr int kMost = (1 << 29) / kUnit;
  if (s.units > kMost) s.units = kMost;
  s.lane = -1;
  int before = 0, slots = 0;
#pragma unroll
  for (int c = 0; c < GDN_MAX_LANES / 64; ++c) {
    if (64 * c >= a.lanes || s.lane >= 0) continue;
    const int n = (u[c] + s.units - 1) / s.units, several = n > 1 ? n : 0;
    const int upto = wave_scan_int(n) + before;
    const int slots_upto = wave_scan_int(several) + slots;
    const bool mine = of_lane ? 64 * c + l == item : upto > item;
    const uint64_t hit = __ballot(mine);
    if (hit) {
      const int w = __builtin_ctzll(hit);
      s.lane = 64 * c + w;
      s.len = __builtin_amdgcn_readlane(len[c], w);
      s.n = __builtin_amdgcn_readlane(n, w);
      s.nth = of_lane ? 0 : item - (__builtin_amdgcn_readlane(upto, w) - s.n);
      s.slot = __builtin_amdgcn_readlane(slots_upto - several, w);
    }
    before = __builtin_amdgcn_readlane(upto, 63);
    slots = __builtin_amdgcn_readlane(slots_upto, 63);
  }
  return s;
}

// ------------------------------------------------------------------ attention
struct AttendArgs {
  KvArgs kv;
  const void* q;
  float* o;
  float* part_o;  // [slots][h_kv][rows][d]
  float* part_ml; // [slots][h_kv][rows][2]: maximum, sum
  float scale;    // of the scores, times log2 e
  int target, rows, groups;  // rows = t_max * h_q / h_kv; row groups of them
};

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float elem(const uint16_t* p, long i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}
__device__ __forceinline__ float elem(const float* p, long i) { return p[i]; }

// The rows of a key-value head are those of q that read it: token t and query
// head h' of its group are row t * group + h'.  Per step of 32 positions a
// wave forms S^T = K Q^T for 16 RT rows, whose result layout (lane column =
// row of q) is at once the B operand of O^T = V^T P^T; V passes through LDS
// for the transposed read.  So the running maximum m and sum l of the softmax
// and the rescaling of O are per lane.  m is raised only when a score is more
// than 2^8 above it, which keeps the exchange between lanes out of nearly
// every step and costs f32 no precision; l stays apart per lane group until
// the end.  P enters as three exact bf16 parts (gdn_mfma_op.h).
//
// Two kernels share this.  For up to 32 rows (16 at D = 256) the four waves
// of attend_kernel share out the positions and each loads its own: the work
// is reading the cache.  For more rows the waves of rows_kernel take 16 rows
// each of the same positions, staged once for all of them.
constexpr float kSlack = 8.f;

// Scores, softmax state and outputs of a wave.
template <int D, typename T, int RT>
struct Rows {
  typedef Op<T> O;
  typedef typename O::Raw Raw;
  typedef typename O::Wide Wide;
  typedef Tile<T, D> TL;        // q and K
  typedef Tile<T, D, true> VL;  // V
  static constexpr int KS = D / 32, CT = D / 16;
  f32x4 acc[RT][CT], sc[RT][2];
  float m[RT], l[RT];
  int end[RT];  // positions that the lane's rows see

  __device__ __forceinline__ void init(int row0, int rows, int len, int T_n,
                                       int group) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int row = row0 + 16 * r + (threadIdx.x & 15);
      end[r] = row < rows ? len - T_n + row / group + 1 : 0;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  // Scores of positions p0 .. p0 + 31 -> sc = exp2(x - m), raising m when
  // needed.  Unless all rows see all of them (whole), bit i of ok says that
  // position p0 + i is in the cache.
  __device__ __forceinline__ void softmax(float scale, bool whole, uint32_t ok,
                                          int p0) {
    const int g4 = (threadIdx.x & 63) >> 4;
    bool raise = false;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[r][h][e] * scale;
          if (!whole) {
            const int i = 16 * h + 4 * g4 + e;
            if (!(ok >> i & 1) || p0 + i >= end[r]) x = -INFINITY;
          }
          sc[r][h][e] = x;
          raise |= x > m[r] + kSlack;
        }
    if (__any(raise)) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float top = m[r];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, sc[r][h][e]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float keep =
            m[r] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[r] - top);
        m[r] = top;
        l[r] *= keep;
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] *= keep;
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float ref = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[r][h][e] = __builtin_amdgcn_exp2f(sc[r][h][e] - ref);
          l[r] += sc[r][h][e];
        }
    }
  }
  // O^T += V^T P^T with V rows r0 .. r0 + 31 of the tile.
  __device__ __forceinline__ void values(const T* Vs, int r0) {
    Wide pw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) pw[r] = O::wide(sc[r][0], sc[r][1]);
    constexpr int kTwo = RT == 1 ? 2 : 1;  // two accumulators at least
#pragma unroll
    for (int c = 0; c < CT; c += kTwo) {
      Raw vf[kTwo];
#pragma unroll
      for (int y = 0; y < kTwo; ++y)
        vf[y] = O::template column<VL>(Vs, r0, 16 * (c + y), 4,
                                       threadIdx.x & 63);
#pragma unroll
      for (int i = 0; i < O::kSteps; ++i)
#pragma unroll
        for (int y = 0; y < kTwo; ++y)
#pragma unroll
          for (int r = 0; r < RT; ++r)
            acc[r][c + y] = O::step(i, vf[y], pw[r], acc[r][c + y]);
    }
  }
  // What infinities and NaN in V at the positions of a step from p0 on add to
  // the rows that see them; `values` took them as zeros.  Rarely needed and
  // slow.
  __device__ __forceinline__ void special(const KvArgs& a, int n, int hk,
                                          int p0, int stop) {
    // (through an empty asm, or what follows from it is kept in registers
    // through the caller's loop)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int g4 = lane >> 4;
    if (stop > p0 + 32) stop = p0 + 32;
#pragma unroll 1
    for (int pos = p0; pos < stop; ++pos) {
      const long row = row_of(a, n, hk, pos, D);
      if (row < 0) continue;
      const int i = pos - p0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float p = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i == (i & 12) + 16 * h + e)  // (uniform)
              p = __shfl(sc[r][h][e], 4 * (i & 12) + (lane & 15));
        const bool sees = pos < end[r];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = elem((const T*)a.v, row + 16 * c + 4 * g4 + e);
            if (sees && !(fabsf(v) < INFINITY)) acc[r][c][e] += p * v;
          }
          __builtin_amdgcn_sched_barrier(0);  // few loads at a time
        }
      }
    }
  }
  // Sums l.  The wave's steps were those of 32 positions from p0, p0 + stride,
  // .. on, before stop.  A row whose m is still -inf has seen no position
  // (l = 0), or scores of -inf alone, which have no softmax: l = 1 then.  Told
  // apart here, where it costs the steps nothing (a count there made windows
  // of 16 1 % slower).
  __device__ __forceinline__ void finish(const KvArgs& a, const int* table,
                                         int p0, int stride, int stop) {
    bool open = false;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      l[r] += __shfl_xor(l[r], 16);
      l[r] += __shfl_xor(l[r], 32);
      open |= m[r] == -INFINITY && p0 < end[r];
    }
    if (!__any(open)) return;
    int first = stop;  // first position that is there
#pragma unroll 1
    for (; p0 < stop && first == stop; p0 += stride) {
      const int pos = p0 + (threadIdx.x & 31);
      const bool there =
          pos < stop && (unsigned)table[page_of(a, pos)] < (unsigned)a.n_pages;
      const uint32_t hit = (uint32_t)__ballot(there);
      if (hit) first = p0 + __builtin_ctz(hit);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
      if (m[r] == -INFINITY && first < stop && first < end[r]) l[r] += 1.f;
  }
};

// q rows row0 .. row0 + n - 1 of a key-value head (zeros past the last).
template <int D, typename T>
__device__ __forceinline__ void stage_q(T* Qs, const AttendArgs& p, int lane,
                                        int hk, int row0, int n, int rows) {
  typedef Tile<T, D> TL;
  const int group = p.kv.h_q / p.kv.h_kv;
  for (int i = threadIdx.x; i < n * TL::kPieces; i += blockDim.x) {
    const int r = i / TL::kPieces, c = i % TL::kPieces;
    u32x4 x = {0, 0, 0, 0};
    if (row0 + r < rows) {
      const int t = (row0 + r) / group, h = hk * group + (row0 + r) % group;
      x = *reinterpret_cast<const u32x4*>(
          (const T*)p.q +
          (((long)lane * p.kv.t_max + t) * p.kv.h_q + h) * D + c * TL::kPer);
    }
    *reinterpret_cast<u32x4*>(Qs + TL::at(r, c)) = x;
  }
}

// Where a row's result goes: o, when the lane has one split, or the split's
// slot (unnormalised, with its m and l).  A row that saw nothing (l = 0) gets
// zeros, one that saw scores of -inf alone NaN.
__device__ __forceinline__ float* row_out(const AttendArgs& p, const Split& s,
                                          int hk, int row, int d, float m,
                                          float l, bool first, float& scale) {
  const KvArgs& a = p.kv;
  const int group = a.h_q / a.h_kv;
  if (s.n == 1) {
    scale = l == 0.f ? 0.f : m == -INFINITY ? NAN : 1.f / l;
    return p.o + (((long)s.lane * a.t_max + row / group) * a.h_q + hk * group +
                  row % group) * d;
  }
  const long at = ((long)(s.slot + s.nth) * a.h_kv + hk) * p.rows + row;
  if (first) {
    p.part_ml[2 * at] = m;
    p.part_ml[2 * at + 1] = l;
  }
  scale = 1.f;
  return p.part_o + at * d;
}

// The four waves' results: each scaled to the common maximum, written to LDS
// (a part of `pitch` floats a wave) and added up by all threads.
constexpr int kSumPad = 4;  // a row's floats past D (rows on different banks)
template <int D, typename R, int ROWS>
__device__ __forceinline__ void sum_waves(const AttendArgs& p, const Split& s,
                                          int hk, int rows, const R& x,
                                          float* pool, int pitch,
                                          float (&ml)[4][2][ROWS]) {
  constexpr int kSumPitch = D + kSumPad, RT = ROWS / 16, CT = R::CT;
  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  if (g4 == 0)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      ml[wave][0][16 * r + n] = x.m[r];
      ml[wave][1][16 * r + n] = x.l[r];
    }
  __syncthreads();
  float* sum = pool + wave * pitch;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w][0][16 * r + n]);
    const float keep =
        x.m[r] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x.m[r] - top);
#pragma unroll
    for (int c = 0; c < CT; ++c)
      *reinterpret_cast<f32x4*>(sum + (16 * r + n) * kSumPitch + 16 * c +
                                4 * g4) = x.acc[r][c] * keep;
  }
  __syncthreads();
  const int used = rows < ROWS ? rows : ROWS;
  for (int i = tid; i < used * (D / 4); i += 256) {
    const int row = i / (D / 4), c = i % (D / 4) * 4;
    float top = -INFINITY, tot = 0.f;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w][0][row]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      tot += ml[w][1][row] *
             (top == -INFINITY ? 1.f
                               : __builtin_amdgcn_exp2f(ml[w][0][row] - top));
      y += *reinterpret_cast<const f32x4*>(pool + w * pitch + row * kSumPitch + c);
    }
    float f;
    float* dst = row_out(p, s, hk, row, D, top, tot, c == 0, f);
    *reinterpret_cast<f32x4*>(dst + c) = y * f;
  }
}

// Few rows: four waves share out a split's positions, 32 at a step.  The next
// step's K rows are loaded when this step's scores are done and its V rows
// when V is in LDS, page numbers a step earlier.  Bound by HBM: 32 lanes x 8
// heads x 16k..32k positions of 128, bf16, 3.3 GB in 582 us (5.7 TB/s).  Short
// caches by what comes in turn (8 lanes x 2 heads of 256): 5.3 us with empty
// caches (launch, lengths, search of the split, q), 8 with one step of one
// wave, 10.6 with one of all four and their sum, 11.7 with eight splits.
template <int D, typename T, int RT>
__global__ __launch_bounds__(256, D * sizeof(T) >= 512 ? 1 : 2) void attend_kernel(
    AttendArgs p, gdn::LaneTable tl) {
  typedef Rows<D, T, RT> R;
  typedef typename R::O O;
  typedef typename R::Raw Raw;
  typedef typename R::TL TL;
  typedef typename R::VL VL;
  constexpr int KS = R::KS, kRows = 16 * RT;
  constexpr int kPieces = sizeof(Raw) / 16;  // 16-byte loads per fragment
  constexpr int kTileBytes = 32 * TL::kPitch * (int)sizeof(T);
  constexpr int kSumBytes = kRows * (D + kSumPad) * 4;
  constexpr int kPer = kTileBytes > kSumBytes ? kTileBytes : kSumBytes;
  __shared__ __attribute__((aligned(16))) T Qs[kRows * TL::kPitch];
  __shared__ __attribute__((aligned(16))) char pool[4 * kPer];
  __shared__ float ml[4][2][kRows];
  const KvArgs& a = p.kv;
  const Split s = find_split(a, tl, blockIdx.x / a.h_kv, p.target, false);
  if (s.lane < 0) return;
  const int hk = blockIdx.x % a.h_kv;
  const int group = a.h_q / a.h_kv, T_n = tl.v[s.lane];
  const int rows = T_n * group;
  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int begin = s.nth * s.units * kUnit;
  const int stop = begin + s.units * kUnit < s.len ? begin + s.units * kUnit : s.len;
  const int steps = (stop - begin + 31) / 32;
  const int open = s.len - T_n + 1;  // first position that some row cannot see
  T* Vs = reinterpret_cast<T*>(pool + wave * kPer);
  const T* kc = (const T*)a.k + 8 * g4;
  const T* vc = (const T*)a.v + 8 * g4;
  const int* table = a.table + (long)s.lane * a.max_pages;

  // position of half h of a step's rows in this lane
  auto pos_of = [&](int step, int h) { return begin + 32 * step + 16 * h + n; };
  int page[2];    // page numbers of the step after the next
  bool there[2];  // whether the rows of the step in hand are
  long at[2];     // and where
  auto look_up = [&](int step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pos = pos_of(step, h);
      page[h] = pos < stop ? table[page_of(a, pos)] : -1;
    }
  };
  auto place = [&](int step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pos = pos_of(step, h);
      const long row = row_in(a, page[h], hk, pos - page_of(a, pos) * a.page, D);
      there[h] = row >= 0;
      at[h] = there[h] ? row : 0;  // (any row of the cache will do)
    }
  };
  u32x4 kr[2][KS][kPieces], vr[2][KS][kPieces];
  auto fetch = [&](const T* c, u32x4 (&r)[2][KS][kPieces]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int x = 0; x < kPieces; ++x)
          r[h][i][x] =
              *reinterpret_cast<const u32x4*>(c + at[h] + 32 * i + 4 * x);
  };

  if (wave < steps) look_up(wave);
  stage_q<D, T>(Qs, p, s.lane, hk, 0, kRows, rows);
  if (wave < steps) {
    place(wave);
    fetch(kc, kr);
    fetch(vc, vr);
    look_up(wave + 4);
  }
  R x;
  x.init(0, rows, s.len, T_n, group);
  __syncthreads();
  for (int step = wave; step < steps; step += 4) {
    const bool here[2] = {there[0], there[1]};
#pragma unroll
    for (int r = 0; r < RT; ++r)
      x.sc[r][0] = x.sc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const Raw qf = O::template row<TL>(Qs, 16 * r, n, 4 * i + g4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Raw kf;
          __builtin_memcpy(&kf, kr[h][i], sizeof(Raw));
          x.sc[r][h] = O::mul(kf, qf, x.sc[r][h]);
        }
      }
    const int next = step + 4;
    if (next < steps) {
      place(next);
      fetch(kc, kr);
      look_up(next + 4);
    }
    const int p0 = begin + 32 * step;
    const bool whole =
        p0 + 32 <= (open < stop ? open : stop) && __all(here[0] && here[1]);
    uint32_t ok = 0;  // bit of position i of the step: its row is there
    if (!whole)
      ok = ((uint32_t)__ballot(here[0]) & 0xffffu) |
           ((uint32_t)__ballot(here[1]) & 0xffffu) << 16;
    x.softmax(p.scale, whole, ok, p0);
    // V through LDS.  Rows that are not there count as zeros.
    if (!whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (!here[h])
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int y = 0; y < kPieces; ++y) vr[h][i][y] = u32x4{0, 0, 0, 0};
    }
    Special<T> odd;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int y = 0; y < kPieces; ++y) odd.look(vr[h][i][y]);
    const bool is_odd = __any(odd.any());
    if (is_odd) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int y = 0; y < kPieces; ++y)
            vr[h][i][y] = Special<T>::cleared(vr[h][i][y]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int y = 0; y < kPieces; ++y)
          *reinterpret_cast<u32x4*>(
              Vs + VL::at(n, kPieces * (4 * i + g4) + y) + 16 * h * VL::kPitch) =
              vr[h][i][y];
    if (next < steps) fetch(vc, vr);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    x.values(Vs, 0);
    if (is_odd) x.special(a, s.lane, hk, p0, stop);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }

  x.finish(a, table, begin + 32 * wave, 128, stop);
  sum_waves<D>(p, s, hk, rows, x, reinterpret_cast<float*>(pool), kPer / 4, ml);
}

// Many rows: NW waves take 16 rows each, and a tile of positions is staged in
// LDS for all of them.  (Four waves of 32 rows read half as much from LDS,
// but two waves per SIMD leave the chain scores - softmax - values exposed: 83
// against 77 us for 8 lanes x 4 heads x 8k..16k positions, 128 rows.  Vector
// ALUs are 58 % busy there, LDS 45 %, matrix cores 37 %.)
template <int D, typename T, int NW>
__global__ __launch_bounds__(64 * NW, D * sizeof(T) >= 512 ? NW / 4 : NW / 2)
void rows_kernel(AttendArgs p, gdn::LaneTable tl) {
  typedef Rows<D, T, 1> R;
  typedef typename R::O O;
  typedef typename R::Raw Raw;
  typedef typename R::TL TL;
  typedef typename R::VL VL;
  constexpr int KS = R::KS, CT = R::CT, kRows = 16 * NW;
  constexpr int kTile = sizeof(T) == 2 ? 64 : 32;  // positions per tile
  constexpr int kStep = 64 * NW / TL::kPieces;     // rows per piece of a thread
  constexpr int kN = kTile / kStep;                // pieces of a thread
  static_assert(kN >= 1 && kN * kStep == kTile, "every thread has a piece");
  __shared__ __attribute__((aligned(16))) T Qs[kRows * TL::kPitch];
  __shared__ __attribute__((aligned(16))) T Ks[kTile * TL::kPitch];
  __shared__ __attribute__((aligned(16))) T Vs[kTile * TL::kPitch];
  __shared__ int odd_tile[2];  // whether a tile's V holds special values
  const KvArgs& a = p.kv;
  const int per_item = a.h_kv * p.groups;
  const Split s = find_split(a, tl, blockIdx.x / per_item, p.target, false);
  if (s.lane < 0) return;
  const int hk = blockIdx.x % per_item / p.groups;
  const int row0 = blockIdx.x % p.groups * kRows;
  const int group = a.h_q / a.h_kv, T_n = tl.v[s.lane];
  const int rows = T_n * group;
  if (row0 >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = gdn::uniform(tid >> 6);
  const int n = lane & 15, g4 = lane >> 4;
  const int begin = s.nth * s.units * kUnit;
  const int stop = begin + s.units * kUnit < s.len ? begin + s.units * kUnit : s.len;
  const int tiles = (stop - begin + kTile - 1) / kTile;
  const int open = s.len - T_n + 1;
  const int* table = a.table + (long)s.lane * a.max_pages;

  // lane i of every wave keeps track of row i of a tile
  int page = -1;        // page number of the row, a tile ahead of its use
  long at = 0;          // where it is
  uint64_t ok = 0;      // rows of the tile in transit that are there
  auto look_up = [&](int tile) {
    const int pos = begin + tile * kTile + lane % kTile;
    page = pos < stop ? table[page_of(a, pos)] : -1;
  };
  auto place = [&](int tile) {
    const int pos = begin + tile * kTile + lane % kTile;
    const long row = row_in(a, page, hk, pos - page_of(a, pos) * a.page, D);
    ok = __ballot(row >= 0);
    at = row >= 0 ? row : 0;
  };
  u32x4 kr[kN], vr[kN];
  const int piece = tid % TL::kPieces, r0 = tid / TL::kPieces;
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int src = r0 + i * kStep;
      const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)at, src);
      const uint32_t hi = (uint32_t)__shfl((int)(at >> 32), src);
      const long off = (long)((uint64_t)hi << 32 | lo) + piece * TL::kPer;
      kr[i] = *reinterpret_cast<const u32x4*>((const T*)a.k + off);
      vr[i] = *reinterpret_cast<const u32x4*>((const T*)a.v + off);
    }
  };
  if (tiles > 0) look_up(0);
  stage_q<D, T>(Qs, p, s.lane, hk, row0, kRows, rows);
  if (tiles > 0) {
    place(0);
    fetch();
    look_up(1);
  }
  R x;
  x.init(row0 + 16 * wave, rows, s.len, T_n, group);
  if (tid == 0) odd_tile[0] = 0;
  for (int tile = 0; tile < tiles; ++tile) {
    const int t0 = begin + tile * kTile;
    const uint64_t here = ok;
    const bool whole = t0 + kTile <= (open < stop ? open : stop) && here == ~0ull;
    __syncthreads();  // the tile before has been read
    Special<T> odd;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = r0 + i * kStep;
      if (!whole && !(here >> r & 1)) vr[i] = u32x4{0, 0, 0, 0};
      odd.look(vr[i]);
    }
    if (odd.any()) {
      odd_tile[tile & 1] = 1;
#pragma unroll
      for (int i = 0; i < kN; ++i) vr[i] = Special<T>::cleared(vr[i]);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      *reinterpret_cast<u32x4*>(Ks + TL::at(r0 + i * kStep, piece)) = kr[i];
      *reinterpret_cast<u32x4*>(Vs + VL::at(r0 + i * kStep, piece)) = vr[i];
    }
    __syncthreads();
    const bool is_odd = odd_tile[tile & 1];
    if (tid == 0) odd_tile[~tile & 1] = 0;
    if (tile + 1 < tiles) {
      place(tile + 1);
      fetch();
      look_up(tile + 2);
    }
    if (row0 + 16 * wave >= rows) continue;
#pragma unroll 1
    for (int half = 0; half < kTile / 32; ++half) {
      x.sc[0][0] = x.sc[0][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const Raw qf = O::template row<TL>(Qs, 16 * wave, n, 4 * i + g4);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x.sc[0][h] = O::mul(
              O::template row<TL>(Ks, 32 * half + 16 * h, n, 4 * i + g4), qf,
              x.sc[0][h]);
      }
      const int p0 = t0 + 32 * half;
      x.softmax(p.scale, whole, (uint32_t)(here >> (32 * half)), p0);
      x.values(Vs, 32 * half);
      if (is_odd) x.special(a, s.lane, hk, p0, stop);
    }
  }
  x.finish(a, table, begin, 32, stop);
  const int row = row0 + 16 * wave + n;
  if (row >= rows) return;
  float f;
  float* dst = row_out(p, s, hk, row, D, x.m[0], x.l[0], g4 == 0, f);
#pragma unroll
  for (int c = 0; c < CT; ++c)
    *reinterpret_cast<f32x4*>(dst + 16 * c + 4 * g4) = x.acc[0][c] * f;
}

// Joins the splits of a lane: a workgroup of NW waves per row of q.  The
// threads first turn the splits' maxima and sums into weights in LDS; then
// each group of D / 4 lanes adds up splits of its own, four columns a lane,
// and the groups' sums meet in registers and LDS.  Bound by its launch and the
// chain length - maxima - partial results, or by reading those.
// One wave per row where there are kManyRows of them (4096 rows of 15 splits:
// 8.7, 9.5, 12.4, 37 us with 1, 2, 4, 16 waves).  Else 4 waves where a lane
// has at most kFewSplits splits, and 16 where it may have more: one lane's
// 25k positions, which are 198 splits, take 13 us with the attention itself,
// against 41 us joined by one wave per row; 4 lanes x 2 heads 31 against 61.
constexpr unsigned kManyRows = 1024;
constexpr int kFewSplits = 64;
constexpr int kFewBlocks = 2048;  // (see shape_of: a lane's splits are no more)
template <int D, int NW, int N>
__global__ __launch_bounds__(64 * NW) void join_kernel(AttendArgs p,
                                                       gdn::LaneTable tl) {
  constexpr int G = D / 4, kSets = 64 * NW / G;  // groups of lanes
  constexpr int kAhead = 4;                      // splits in flight per group
  __shared__ float weight[N];
  __shared__ float tops[NW], sums[NW];
  __shared__ __attribute__((aligned(16))) f32x4 part[NW][G];
  const KvArgs& a = p.kv;
  const int per_lane = a.h_kv * p.rows;
  const int n = (int)(blockIdx.x / per_lane), at = (int)(blockIdx.x % per_lane);
  const int hk = at / p.rows, row = at % p.rows;
  const int group = a.h_q / a.h_kv;
  if (row >= tl.v[n] * group) return;
  const Split s = find_split(a, tl, n, p.target, true);
  if (s.n < 2) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int set = tid / G, c = tid % G * 4;
  const long first = ((long)s.slot * a.h_kv + hk) * p.rows + row;
  const long step = (long)a.h_kv * p.rows;
  const float* src = p.part_o + first * D + c;
  f32x4 y[kAhead];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * kSets;
      y[u] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i < s.n)
        y[u] = *reinterpret_cast<const f32x4*>(src + i * step * D);
    }
  };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + first;
  // a thread's first split is kept, further ones are read again
  float2 mine = {-INFINITY, 0.f};
  if (tid < s.n) mine = ml[tid * step];
  fetch(set);
  float m = mine.x, l = 0.f;
  for (int i = tid + 64 * NW; i < s.n; i += 64 * NW)
    m = fmaxf(m, ml[i * step].x);
#pragma unroll
  for (int x = 1; x < 64; x *= 2) m = fmaxf(m, __shfl_xor(m, x));
  if (lane == 0) tops[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < NW; ++w) m = fmaxf(m, tops[w]);
  for (int i = tid; i < s.n; i += 64 * NW) {
    if (i != tid) mine = ml[i * step];
    // (a split that saw nothing has no weight, one with a NaN keeps it, and
    // where all that was seen scored -inf the weights are NaN)
    const float w = mine.x == -INFINITY && mine.y == 0.f
                        ? 0.f
                        : __builtin_amdgcn_exp2f(mine.x - m);
    weight[i] = w;
    l = __builtin_fmaf(w, mine.y, l);
  }
  l = gdn::wave_sum(l);
  if (lane == 0) sums[wave] = l;
  __syncthreads();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = set; i0 < s.n; i0 += kAhead * kSets) {
    if (i0 != set) fetch(i0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u * kSets < s.n) acc += y[u] * weight[i0 + u * kSets];
  }
#pragma unroll
  for (int x = G; x < 64; x *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], x);
  if (lane < G) part[wave][lane] = acc;
  __syncthreads();
  if (tid >= G) return;
  l = 0.f;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    l += sums[w];
    acc += part[w][tid];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float* dst = p.o + (((long)n * a.t_max + row / group) * a.h_q + hk * group +
                      row % group) * D;
  *reinterpret_cast<f32x4*>(dst + c) = acc * inv;
}

// One 16-byte piece of a key and of a value row per thread: a copy (8,192 rows
// of 8 heads, 67 MB in 14 us), or its launch.
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
  const long pos = (long)a.kv_len[n] - T + t;
  if (pos < 0 || pos >= a.max_pages * a.page) return;
  const long dst = row_of(a, n, h, (int)pos, pieces);
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
      (double)d.max_pages * d.page_size >= (double)(1 << 29) ||
      (double)d.n_lanes * d.t_max * d.h_q * 32 > (double)INT_MAX ||
      (double)d.n_lanes * d.h_q * 1024 > (double)INT_MAX ||
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
  KvArgs a = {k,     v,      table,       kv_len,    d.n_lanes,   d.t_max,
              d.h_q, d.h_kv, d.page_size, d.n_pages, d.max_pages, 0u, 0};
  // division by the page size for positions below 2^30 (with 2^s >= page,
  // multiplier floor(2^32 (2^s - page) / page) + 1)
  while ((1l << a.page_shift) < d.page_size) ++a.page_shift;
  a.page_mul = (uint32_t)(((uint64_t)((1l << a.page_shift) - d.page_size) << 32) /
                              (uint64_t)d.page_size +
                          1);
  return a;
}

// How a call is spread: few rows of q (attend_kernel) or many in groups of
// 16 a wave (rows_kernel), and the splits: kFewBlocks and kRowsBlocks workgroups
// in all, short last splits included, and no more than the page tables have
// units.  Measured, for 32 lanes x 8 heads x 16k..32k positions, one token:
// 780, 618, 588, 584 us with 512, 1024, 1536, 2048 workgroups (more of them
// even out the memory's latency); for 8 lanes x 4 heads x 8k..16k, 128 rows:
// 121, 93, 117, 110 us with 256, 512, 768, 1024 (two a CU run at once there,
// d = 128 in bf16, and every split of 128 rows leaves 64 KiB to join; d = 256,
// and d = 128 in f32 with eight waves, fit one a CU and take the same number
// without a measurement of their own).  Rows of 512 bytes and more
// leave one workgroup of attend_kernel per CU, whose start and end nothing
// hides, so there are as many as CUs (kWideBlocks): d = 256, bf16, 2 heads, 8
// lanes x 4k..8k: 32, 37, 37, 49, 49 us with 256, 512, 768, 1024, 2048; one
// lane x 30k: 23 us, and 30 with any more; 66 lanes x up to 8.5k: 102, 106,
// 108, 119, 128 us; f32, d = 128, 16 lanes x 8 heads: 124, 105, 102, 109, 119.
constexpr int kRowsBlocks = 512;
constexpr int kWideBlocks = 256;

struct Shape {
  int rows, rt, waves, groups, target, items, slots;
  bool few;
};
static Shape shape_of(const gdn_kv_dims& d, int few_blocks, int rows_blocks) {
  Shape s;
  s.rows = d.t_max * (d.h_q / d.h_kv);
  s.few = s.rows <= (d.d < 256 ? 32 : 16);
  s.rt = s.few && s.rows > 16 ? 2 : 1;
  s.waves = !s.few && s.rows > 64 && d.d < 256 ? 8 : 4;
  s.groups = s.few ? 1 : (s.rows + 16 * s.waves - 1) / (16 * s.waves);
  const int blocks = s.few ? few_blocks : rows_blocks;
  const int items = blocks / (d.h_kv * s.groups);
  s.target = items - d.n_lanes > items / 2 ? items - d.n_lanes : items / 2;
  if (s.target < 1) s.target = 1;
  const long units = ((long)d.max_pages * d.page_size + kUnit - 1) / kUnit;
  const long most = units * d.n_lanes;
  s.items = s.target + d.n_lanes < most ? s.target + d.n_lanes : (int)most;
  s.slots = 2l * s.target < most ? 2 * s.target : (int)most;
  return s;
}
static Shape shape_of(const gdn_kv_dims& d, int size) {
  return shape_of(d, d.d * size < 512 ? kFewBlocks : kWideBlocks, kRowsBlocks);
}
static size_t slot_bytes(const gdn_kv_dims& d, const Shape& s) {
  const size_t n = (size_t)s.slots * d.h_kv * s.rows;
  return n * (d.d + 2) * sizeof(float);
}
// (bf16 never needs less)
static size_t attend_bytes(const gdn_kv_dims& d) {
  return slot_bytes(d, shape_of(d, 2));
}

// MOST: waves that join one row where there are few rows and many splits.
template <int D, int MOST = 16>
static hipError_t join(const gdn_kv_dims& d, const Shape& s,
                       const AttendArgs& p, const gdn::LaneTable& tl,
                       hipStream_t st) {
  // a cache of one unit per lane has nothing to join
  const long units = ((long)d.max_pages * d.page_size + kUnit - 1) / kUnit;
  if (units < 2) return hipSuccess;
  const dim3 rows((unsigned)((long)d.n_lanes * d.h_kv * s.rows));
  if (rows.x >= kManyRows)
    return launch(join_kernel<D, 1, kFewBlocks>, rows, dim3(64), st, p, tl);
  if (units <= kFewSplits || s.target <= kFewSplits)
    return launch(join_kernel<D, 4, kFewSplits>, rows, dim3(256), st, p, tl);
  return launch(join_kernel<D, MOST, kFewBlocks>, rows, dim3(64 * MOST), st, p, tl);
}

template <int D, typename T>
static hipError_t attend(const gdn_kv_dims& d, const Shape& s,
                         const AttendArgs& p, const gdn::LaneTable& tl,
                         hipStream_t st) {
  const dim3 grid((unsigned)((long)s.items * d.h_kv * s.groups));
  hipError_t e;
  if constexpr (D < 256) {
    if (s.few)
      e = s.rt == 2 ? launch(attend_kernel<D, T, 2>, grid, dim3(256), st, p, tl)
                    : launch(attend_kernel<D, T, 1>, grid, dim3(256), st, p, tl);
    else
      e = s.waves == 8
              ? launch(rows_kernel<D, T, 8>, grid, dim3(512), st, p, tl)
              : launch(rows_kernel<D, T, 4>, grid, dim3(256), st, p, tl);
  } else {
    e = s.few ? launch(attend_kernel<D, T, 1>, grid, dim3(256), st, p, tl)
              : launch(rows_kernel<D, T, 4>, grid, dim3(256), st, p, tl);
  }
  return e != hipSuccess ? e : join<D>(d, s, p, tl, st);
}

template <typename T>
static hipError_t attend(const gdn_kv_dims& d, const Shape& s,
                         const AttendArgs& p, const gdn::LaneTable& tl,
                         hipStream_t st) {
  if (d.d == 64) return attend<64, T>(d, s, p, tl, st);
  if (d.d == 128) return attend<128, T>(d, s, p, tl, st);
  return attend<256, T>(d, s, p, tl, st);
}

}  // namespace gdnk

extern "C" size_t gdn_paged_attention_workspace_bytes(const gdn_kv_dims* dims) {
  if (gdnk::check_kv_dims("gdn_paged_attention_workspace_bytes", dims) !=
      GDN_OK)
    return 0;
  return gdnk::attend_bytes(*dims);
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
  const Shape s = shape_of(*dims, dtype == GDN_BF16 ? 2 : 4);
  AttendArgs p;
  p.kv = kv_args(*dims, k_cache, v_cache, page_table, kv_len);
  p.q = q;
  p.o = o;
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + (size_t)s.slots * dims->h_kv * s.rows * dims->d;
  p.scale = scale * kLog2e;
  p.target = s.target;
  p.rows = s.rows;
  p.groups = s.groups;
  const hipError_t e =
      dtype == GDN_BF16
          ? attend<uint16_t>(*dims, s, p, tl, (hipStream_t)stream)
          : attend<float>(*dims, s, p, tl, (hipStream_t)stream);
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
