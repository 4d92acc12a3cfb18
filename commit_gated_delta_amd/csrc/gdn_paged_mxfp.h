// gdn_paged_mxfp.h -- attention of draft windows or single tokens over a paged
// key-value cache held in 4 bits (gdn_paged_attention_mxfp).  Compiled as part
// of gdn_state.hip.
//
// The splits, the softmax and the layout of scores and outputs are those of
// gdn_paged.h; what differs is how K and V reach the matrix cores:
//
// Scores.  A product may sum its slots in any order, so a lane takes a quarter
// of a row's channels as they lie in the cache, and each dword of codes,
// widened to bf16 (exact), is its part of an operand of 16 x 16 x 32 against
// the same channels of q.  (The instructions that take 4-bit codes and their
// scales as they are multiply by 8-bit floats at most, and add up with about
// 16 bits below the largest product: q cut into two or five such floats gave
// log probabilities 5e-6 off, rms, where this gives 1e-7.)
//
// Values are widened on their way through LDS, from where the transposed read
// takes them as in gdn_paged.h.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_mxfp.h"
#include "gdn_paged.h"

namespace gdnk {

struct Attend4Args {
  AttendArgs at;  // (its scale without its sign)
  Fp4Rows k4, v4;
  uint32_t flip;  // turns the signs of a dword of q, where the scale is negative
};

// What lane 16 g + n holds of a row: its channels D / 4 g .. D / 4 (g + 1) - 1,
// so of codes D / 32 dwords, each an operand's eight slots, in one or two
// blocks.
template <int D>
struct Own {
  static constexpr int kDwords = D / 32;
  static constexpr int kScales = D == 256 ? 2 : 1;
  uint32_t codes[kDwords];
  uint32_t scale[kScales];
  // Of row `row` + `more`, which may be the wave's and the lane's part.
  __device__ __forceinline__ void load(const Fp4Rows& c, uint32_t row,
                                       uint32_t more, int g) {
    const uint8_t* at = c.codes + (uint64_t)row * (D / 2) +
                        (more * (D / 2) + (D / 8) * g);
    if constexpr (D == 64) {
      const uint2 w = *reinterpret_cast<const uint2*>(at);
      codes[0] = w.x;
      codes[1] = w.y;
    } else {
#pragma unroll
      for (int y = 0; y < kDwords / 4; ++y) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(at + 16 * y);
#pragma unroll
        for (int i = 0; i < 4; ++i) codes[4 * y + i] = w[i];
      }
    }
    const uint8_t* s = c.scales + (uint64_t)row * (D / 32);
    if constexpr (D == 256) {
      const uint32_t w =
          *reinterpret_cast<const uint16_t*>(s + (more * (D / 32) + 2 * g));
      scale[0] = w & 255;
      scale[1] = w >> 8;
    } else {
      scale[0] = s[more * (D / 32) + (D == 64 ? g >> 1 : g)];
    }
  }
  __device__ __forceinline__ bool odd() const {  // whether a block is NaN
    const uint32_t x = scale[0], y = scale[kScales - 1];
    return (x > y ? x : y) >= kScaleOdd;
  }
  __device__ __forceinline__ u32x4 values(int i) const {
    return fp4_values(codes[i], scale[i * kScales / kDwords]);
  }
};

// Query rows as B operands: lane 16 g + n holds channels D / 4 g + 8 i .. + 7
// of row n, i < D / 32; f32 rows as three bf16 parts.
template <int D, typename T>
struct Query {
  typedef Op<uint16_t> O;
  typedef std::conditional_t<sizeof(T) == 2, u32x4, typename O::Wide> Piece;
  Piece q[D / 32];
  // The row at `row`, its signs turned by `flip`, or zeros.
  __device__ __forceinline__ void load(const T* row, uint32_t flip, bool zero) {
    const T* at = row + (D / 4) * ((threadIdx.x & 63) >> 4);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      u32x4 w[sizeof(T) / 2];
#pragma unroll
      for (int y = 0; y < (int)sizeof(T) / 2; ++y) {
        w[y] = reinterpret_cast<const u32x4*>(at + 8 * i)[y] ^ flip;
        if (zero) w[y] = u32x4{0, 0, 0, 0};
      }
      if constexpr (sizeof(T) == 2) q[i] = w[0];
      else q[i] = O::wide(__builtin_bit_cast(f32x4, w[0]), __builtin_bit_cast(f32x4, w[1]));
    }
  }
};

// Scores of twice 16 positions against RT times 16 rows.
template <int D, typename T, int RT>
__device__ __forceinline__ void scores_of(const Own<D> (&k)[2],
                                          const Query<D, T> (&q)[RT],
                                          f32x4 (&c)[RT][2]) {
  typedef Op<uint16_t> O;
#pragma unroll
  for (int r = 0; r < RT; ++r) c[r][0] = c[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const u32x4 a = k[0].values(i), b = k[1].values(i);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if constexpr (sizeof(T) == 2) {
        c[r][0] = O::mul(a, q[r].q[i], c[r][0]);
        c[r][1] = O::mul(b, q[r].q[i], c[r][1]);
      } else {
#pragma unroll
        for (int y = 0; y < O::kSteps; ++y) {
          c[r][0] = O::step(y, a, q[r].q[i], c[r][0]);
          c[r][1] = O::step(y, b, q[r].q[i], c[r][1]);
        }
      }
    }
  }
}

// The row of q at row `row` of key-value head hk.
template <int D, typename T>
__device__ __forceinline__ const T* query_row(const AttendArgs& p, int lane,
                                              int hk, int row) {
  const int group = p.kv.h_q / p.kv.h_kv;
  return (const T*)p.q + (((long)lane * p.kv.t_max + row / group) * p.kv.h_q +
                          hk * group + row % group) * D;
}

// A V tile as Tile's, with neighbouring pieces swapped in every other eight
// rows: 16 lanes then write one piece of 16 rows, as they read two of eight,
// without a conflict (13 % of a wave's time at D = 128).
template <int D>
struct VTile {
  typedef Tile<uint16_t, D, true> Base;
  static constexpr int kPitch = Base::kPitch;
  static __device__ __forceinline__ int at(int r, int p) {
    return Base::at(r, p ^ (r >> 3 & 1));
  }
};

// Scores, softmax state and outputs of a wave, as Rows.  The scale is not
// negative here (a query's signs carry that), so the largest of the raw
// scores tells whether m is to be raised, and one operation scales a score
// and subtracts m.
//
// m is rounded, the scaled score in that operation is not, so the largest
// weight is not 1 but 2 to the half step that m is off by: nothing to a
// softmax, whose sum has the same factor, while it is a small power of two.
// With a row past kFar the scaled scores are rounded as m is (in f32, scores of
// that size are whole octaves apart in any case), and m is raised without slack,
// which would be lost in it.  Such a row's lim lets every step through to where
// m is raised, so that the other steps need not ask.  (A raw score of +inf
// needs none of this: it gives NaN in either way.)
constexpr float kFar = 16777216.f;  // 2^24: m is off by one at most
template <int D, int RT>
struct Rows4 : Rows<D, uint16_t, RT> {
  typedef Rows<D, uint16_t, RT> R;
  float lim[RT];   // raw score above which m is raised
  float base[RT];  // what is added to a scaled score: -m, 0 before the first

  __device__ __forceinline__ void init(int row0, int rows, int len, int T_n,
                                       int group) {
    R::init(row0, rows, len, T_n, group);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      lim[r] = -INFINITY;
      base[r] = 0.f;
    }
  }
  // As Rows::softmax, on the raw scores in sc.
  __device__ __forceinline__ void softmax(float scale, bool whole, uint32_t ok,
                                          int p0) {
    const int g4 = (threadIdx.x & 63) >> 4;
    uint32_t sees[RT];  // bit 4 h + e: score [h][e] counts
    if (!whole) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        sees[r] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * h + 4 * g4 + e;
            const bool on = (ok >> i & 1) && p0 + i < this->end[r];
            sees[r] |= on << (4 * h + e);
            if (!on) this->sc[r][h][e] = -INFINITY;
          }
      }
    }
    bool raise = false;
    float top[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const f32x4 a = this->sc[r][0], b = this->sc[r][1];
      top[r] = fmaxf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])),
                     fmaxf(fmaxf(b[0], b[1]), fmaxf(b[2], b[3])));
      raise |= top[r] > lim[r];
    }
    if (__any(raise)) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float t = top[r];
        t = fmaxf(t, __shfl_xor(t, 16));
        t = fmaxf(t, __shfl_xor(t, 32));
        const bool rounds = t < INFINITY && fabsf(t * scale) > kFar;
        t = t == -INFINITY ? t : fmaxf(this->m[r], t * scale);
        if (t > this->m[r]) {
          const float keep = this->m[r] == -INFINITY
                                 ? 0.f
                                 : __builtin_amdgcn_exp2f(this->m[r] - t);
          this->m[r] = t;
          base[r] = -t;
          lim[r] = rounds        ? -INFINITY
                   : scale > 0.f ? (t + kSlack) / scale
                                 : INFINITY;
          this->l[r] *= keep;
#pragma unroll
          for (int c = 0; c < R::CT; ++c) this->acc[r][c] *= keep;
        }
      }
      bool past = false;
#pragma unroll
      for (int r = 0; r < RT; ++r)
        past |= lim[r] == -INFINITY && this->m[r] != -INFINITY;
      if (__any(past)) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) this->sc[r][h] *= scale;
        scale = 1.f;
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          this->sc[r][h][e] = __builtin_amdgcn_exp2f(
              __builtin_fmaf(this->sc[r][h][e], scale, base[r]));
    if (!whole) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(sees[r] >> (4 * h + e) & 1)) this->sc[r][h][e] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const f32x4 a = this->sc[r][0], b = this->sc[r][1];
      this->l[r] += ((a[0] + a[1]) + (a[2] + a[3])) + ((b[0] + b[1]) + (b[2] + b[3]));
    }
  }
  // O^T += V^T P^T with V rows r0 .. r0 + 31 of the tile.
  __device__ __forceinline__ void values(const uint16_t* Vs, int r0) {
    typedef Op<uint16_t> O;
    typename O::Wide pw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
      pw[r] = O::wide(this->sc[r][0], this->sc[r][1]);
    constexpr int kTwo = RT == 1 ? 2 : 1;  // two accumulators at least
#pragma unroll
    for (int c = 0; c < R::CT; c += kTwo) {
      u32x4 vf[kTwo];
#pragma unroll
      for (int y = 0; y < kTwo; ++y)
        vf[y] = O::template column<VTile<D>>(Vs, r0, 16 * (c + y), 4,
                                             threadIdx.x & 63);
#pragma unroll
      for (int i = 0; i < O::kSteps; ++i)
#pragma unroll
        for (int y = 0; y < kTwo; ++y)
#pragma unroll
          for (int r = 0; r < RT; ++r)
            this->acc[r][c + y] = O::step(i, vf[y], pw[r], this->acc[r][c + y]);
    }
  }
};

// Rows that see a position whose value block b is NaN get NaN in its
// channels; `values` took it as zeros.  What a row sees is a prefix, so the
// first such position, p0 + first, is enough.
template <int D, int RT>
__device__ __forceinline__ void mark_odd(Rows4<D, RT>& x, int b,
                                         int pos) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c / 2 == b && pos < x.end[r]) x.acc[r][c][e] = NAN;
}

// Waves per SIMD that the registers are kept to: f32 queries take three times
// the registers of bf16 ones.
template <int D, typename T, int RT>
constexpr int few4_waves() {
  constexpr int q = D * RT * (int)sizeof(T);
  return D * RT == 64 ? 4 : q <= 256 ? 3 : q <= 512 ? 2 : 1;
}
template <int D, typename T, int NW, int RT>
constexpr int rows4_waves() {
  return RT == 2 || D * sizeof(T) > 256 ? NW / 4 * RT : NW / 2;
}
// Whether a wave of rows4_kernel takes 32 rows of 128, so that K is widened
// and V read half as often, or 16 (the same windows of 16 over 16k): 57.1 and
// 59.5 us with the join at d = 64, 72.3 and 78.9 at 128, in f32 61.0 and 63.9
// at 64.  At 128 f32 rows are taken by 16 (104 us): 32 of them take 115 us with
// one wave a SIMD, and 94 with two, which spill 16 registers.
template <int D, typename T>
constexpr bool kWide = D * sizeof(T) <= 256;

// Row of a position in its page, counted over the cache (fewer than 2^32).
__device__ __forceinline__ uint32_t cache_row(const KvArgs& a, int page, int h,
                                              int pos, bool& there) {
  there = (unsigned)page < (unsigned)a.n_pages;
  const uint32_t row = ((uint32_t)page * a.h_kv + h) * a.page +
                       (uint32_t)(pos - page_of(a, pos) * a.page);
  return there ? row : 0;  // (any row of the cache will do)
}

// Few rows, as attend_kernel: four waves share out a split's positions, 32 at
// a step, and lane 16 g + n holds its channels of positions n and 16 + n.
// EVEN: pages are multiples of 16 positions, so that each half of a step lies
// in one page, whose number and place are the wave's and not the lanes'.
//
// A cache of this kind is read once, 17 bytes for 32 channels, so memory is
// what bounds it: 32 lanes of up to 32k positions, 8 heads of 128 under four
// queries each, take 177 us, 5.0 TB/s, where the loads alone take 164.  The
// loads of a step are given out a whole step ahead, each into the registers
// that the step in hand has just used up; with a branch around the last ones
// it was 200 us.  A short cache is bound by one workgroup's chain of look-up,
// loads, products and sums: 8 lanes of up to 1k positions 8.8 us and 4.2 for
// the join.
template <int D, typename T, int RT, bool EVEN>
__global__ __launch_bounds__(256, (few4_waves<D, T, RT>())) void attend4_kernel(
    Attend4Args q, gdn::LaneTable tl) {
  typedef Rows4<D, RT> R;
  typedef VTile<D> VL;
  typedef Own<D> Part;
  constexpr int kRows = 16 * RT;
  constexpr int kTileBytes = 32 * D * 2;
  constexpr int kSumBytes = kRows * (D + kSumPad) * 4;
  constexpr int kWave = kTileBytes > kSumBytes ? kTileBytes : kSumBytes;
  __shared__ __attribute__((aligned(16))) char pool[4 * kWave];
  __shared__ float ml[4][2][kRows];
  const AttendArgs& p = q.at;
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
  uint16_t* Vs = reinterpret_cast<uint16_t*>(pool + wave * kWave);
  const int* table = a.table + (long)s.lane * a.max_pages;

  int page[2];     // page numbers of the step after the next
  bool there[2];   // whether the positions of the step in hand are
  uint32_t at[2];  // and their rows (EVEN: that of the half's first one)
  const uint32_t more = EVEN ? n : 0;
  auto pos_of = [&](int step, int h) {
    return begin + 32 * step + 16 * h + (EVEN ? 0 : n);
  };
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
      at[h] = cache_row(a, page[h], hk, pos, there[h]);
      if (EVEN) there[h] = there[h] && pos + n < stop;
    }
  };
  Part kp[2], vp[2];
  auto fetch = [&](const Fp4Rows& c, Part (&r)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) r[h].load(c, at[h], more, g4);
  };

  // (Past the last step a lane loads the cache's first row: a branch around
  // the loads would have the compiler copy what they return, and wait for it.)
  look_up(wave);
  place(wave);
  fetch(q.k4, kp);
  fetch(q.v4, vp);
  look_up(wave + 4);
  R x;
  x.init(0, rows, s.len, T_n, group);
  Query<D, T> query[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // (rows past the last: the first one's channels as zeros)
    const int row = 16 * r + n < rows ? 16 * r + n : 0;
    query[r].load(query_row<D, T>(p, s.lane, hk, row), q.flip, 16 * r + n >= rows);
  }
  for (int step = wave; step < steps; step += 4) {
    const bool here[2] = {there[0], there[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (__any(kp[h].odd()))
#pragma unroll
        for (int y = 0; y < Part::kScales; ++y)
          if (kp[h].scale[y] >= kScaleOdd) kp[h].scale[y] = kScaleNan;
    }
    scores_of<D, T>(kp, query, x.sc);
    place(step + 4);
    fetch(q.k4, kp);
    look_up(step + 8);
    const int p0 = begin + 32 * step;
    const bool whole =
        p0 + 32 <= (open < stop ? open : stop) && __all(here[0] && here[1]);
    uint32_t ok = 0;  // bit of position i of the step: its row is there
    if (!whole)
      ok = ((uint32_t)__ballot(here[0]) & 0xffffu) |
           ((uint32_t)__ballot(here[1]) & 0xffffu) << 16;
    x.softmax(p.scale, whole, ok, p0);
    // V through LDS.  Rows that are not there and blocks of NaN count as zeros.
    bool off[2][Part::kScales];
    const bool is_odd = __any((here[0] & vp[0].odd()) | (here[1] & vp[1].odd()));
    if (is_odd || !whole) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int y = 0; y < Part::kScales; ++y) {
          off[h][y] = here[h] && vp[h].scale[y] >= kScaleOdd;
          if (off[h][y] || !here[h]) {
            vp[h].scale[y] = 0;
#pragma unroll
            for (int i = 0; i < Part::kDwords; ++i)
              if (i * Part::kScales / Part::kDwords == y) vp[h].codes[i] = 0;
          }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < Part::kDwords; ++i)
        *reinterpret_cast<u32x4*>(Vs + VL::at(n, Part::kDwords * g4 + i) +
                                  16 * h * VL::kPitch) = vp[h].values(i);
    fetch(q.v4, vp);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    x.values(Vs, 0);
    if (is_odd) {
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        // positions of the step whose block b is NaN
        const int y = D == 256 ? b & 1 : 0;
        const int g = D == 64 ? 32 * b : D == 128 ? 16 * b : 16 * (b >> 1);
        const uint32_t hit = ((uint32_t)(__ballot(off[0][y]) >> g) & 0xffffu) |
                             ((uint32_t)(__ballot(off[1][y]) >> g) & 0xffffu) << 16;
        if (hit) mark_odd(x, b, p0 + __builtin_ctz(hit));
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  x.finish(a, table, begin + 32 * wave, 128, stop);
  sum_waves<D>(p, s, hk, rows, x, reinterpret_cast<float*>(pool), kWave / 4, ml);
}

// Many rows, as rows_kernel: NW waves take 16 RT rows each of the same tile of
// 64 positions, whose K lies in LDS as it is in the cache and whose V is
// widened once for all of them.
//
// What a wave does one after the other bounds it: vector instructions 54 % of
// the time (K is widened, each probability cut into the three bf16 parts that
// hold its 24 bits), matrix ones 39 % (four products a score, one for K and
// three for V); two waves a SIMD hide little of either behind the other.  8
// lanes x 16 tokens x 32 heads of 128 over up to 16k positions: 68 us.  With
// 16 rows a wave it was 76; with K widened once for all waves, as V is, 84,
// bound by the reads from LDS; scores of the whole tile before its softmax, or
// a wave's priority raised for its products, change nothing (68..69).
template <int D, typename T, int NW, int RT>
__global__ __launch_bounds__(64 * NW, (rows4_waves<D, T, NW, RT>())) void rows4_kernel(
    Attend4Args q, gdn::LaneTable tl) {
  typedef Rows4<D, RT> R;
  typedef VTile<D> VL;
  constexpr int kRows = 16 * NW * RT, kTile = 64, kBlocks = D / 32;
  constexpr int kPieces = kTile * kBlocks;                    // of K, or of V
  constexpr int kThreads = 64 * NW;
  constexpr int kN = (kPieces + kThreads - 1) / kThreads;     // of a thread
  __shared__ __attribute__((aligned(16))) u32x4 Kc[kPieces];
  __shared__ uint8_t Ks[kPieces];
  __shared__ __attribute__((aligned(16))) uint16_t Vs[kTile * D];
  __shared__ int odd_first[2][kBlocks];  // of a tile's rows, by block; kTile: none
  const AttendArgs& p = q.at;
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
  uint32_t at = 0;      // where it is
  uint64_t ok = 0;      // rows of the tile in transit that are there
  auto look_up = [&](int tile) {
    const int pos = begin + tile * kTile + lane;
    page = pos < stop ? table[page_of(a, pos)] : -1;
  };
  auto place = [&](int tile) {
    bool there;
    at = cache_row(a, page, hk, begin + tile * kTile + lane, there);
    ok = __ballot(there);
  };
  u32x4 kr[kN], vr[kN];
  uint32_t ks[kN], vs[kN];
  // (threads without a piece take a copy of another's)
  auto piece_of = [&](int i) { return (tid + i * kThreads) % kPieces; };
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int src = piece_of(i) / kBlocks, b = piece_of(i) % kBlocks;
      const uint64_t off = (uint64_t)(uint32_t)__shfl((int)at, src) * kBlocks + b;
      kr[i] = *reinterpret_cast<const u32x4*>(q.k4.codes + 16 * off);
      ks[i] = q.k4.scales[off];
      vr[i] = *reinterpret_cast<const u32x4*>(q.v4.codes + 16 * off);
      vs[i] = q.v4.scales[off];
    }
  };
  // Place of block b of row r in Kc and Ks: rows of 2 to 8 blocks share 256
  // bytes, their blocks permuted so that 16 rows' block b lie apart.
  auto spot = [&](int r, int b) {
    return r * kBlocks + (b ^ (r / (16 / kBlocks)) % kBlocks);
  };
  auto put = [&](int tile, uint64_t here) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = piece_of(i) / kBlocks, b = piece_of(i) % kBlocks;
      const bool is_there = here >> r & 1, off = vs[i] >= kScaleOdd;
      if (is_there && off) atomicMin(&odd_first[tile & 1][b], r);
      if (!is_there || off) {
        vr[i] = u32x4{0, 0, 0, 0};
        vs[i] = 0;
      }
      Kc[spot(r, b)] = kr[i];
      Ks[spot(r, b)] = (uint8_t)(ks[i] >= kScaleOdd ? kScaleNan : ks[i]);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        *reinterpret_cast<u32x4*>(Vs + VL::at(r, 4 * b + y)) =
            fp4_values(vr[i][y], vs[i]);
    }
  };
  if (tid < 2 * kBlocks) odd_first[tid / kBlocks][tid % kBlocks] = kTile;
  // (past the last tile, loads of the cache's first row, as in attend4_kernel)
  look_up(0);
  place(0);
  fetch();
  look_up(1);
  R x;
  x.init(row0 + 16 * RT * wave, rows, s.len, T_n, group);
  Query<D, T> query[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = row0 + 16 * (RT * wave + r) + n;
    query[r].load(query_row<D, T>(p, s.lane, hk, row < rows ? row : 0), q.flip,
                  row >= rows);
  }
  for (int tile = 0; tile < tiles; ++tile) {
    const int t0 = begin + tile * kTile;
    const uint64_t here = ok;
    const bool whole = t0 + kTile <= (open < stop ? open : stop) && here == ~0ull;
    __syncthreads();  // the tile before has been read
    put(tile, here);
    place(tile + 1);
    fetch();
    look_up(tile + 2);
    __syncthreads();
    if (tid < kBlocks) odd_first[~tile & 1][tid] = kTile;
    if (row0 + 16 * RT * wave >= rows) continue;
#pragma unroll 1
    for (int half = 0; half < kTile / 32; ++half) {
      Own<D> k[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 32 * half + 16 * h + n;
        if constexpr (D == 64) {
          const int w = spot(r, g4 >> 1);
          const uint2 y = reinterpret_cast<const uint2*>(&Kc[w])[g4 & 1];
          k[h].codes[0] = y.x;
          k[h].codes[1] = y.y;
          k[h].scale[0] = Ks[w];
        } else {
#pragma unroll
          for (int y = 0; y < D / 128; ++y) {
            const int w = spot(r, D / 128 * g4 + y);
            const u32x4 c = Kc[w];
#pragma unroll
            for (int i = 0; i < 4; ++i) k[h].codes[4 * y + i] = c[i];
            k[h].scale[y] = Ks[w];
          }
        }
      }
      scores_of<D, T>(k, query, x.sc);
      const int p0 = t0 + 32 * half;
      x.softmax(p.scale, whole, (uint32_t)(here >> (32 * half)), p0);
      x.values(Vs, 32 * half);
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int first = gdn::uniform(odd_first[tile & 1][b]);
      if (first < kTile) mark_odd(x, b, t0 + first);
    }
  }
  x.finish(a, table, begin, 32, stop);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = row0 + 16 * (RT * wave + r) + n;
    if (row >= rows) return;
    float f;
    float* dst = row_out(p, s, hk, row, D, x.m[r], x.l[r], g4 == 0, f);
#pragma unroll
    for (int c = 0; c < R::CT; ++c)
      *reinterpret_cast<f32x4*>(dst + 16 * c + 4 * g4) = x.acc[r][c] * f;
  }
}

// ---------------------------------------------------------------- host side
// Workgroups of a launch, as kFewBlocks and kRowsBlocks of the wider cache.
// 32 lanes of up to 32k, 8 heads of 128: 280, 198, 197, 176, 177 us with 512,
// 768, 1024, 1536, 2048; f32 queries, 13 lanes of up to 10k, 3 heads of 64:
// 14.4, 14.5, 14.8, 16.0, 15.7 (the long caches decide; a short split is mostly
// its start and end); 8 lanes of up to 1k have fewer splits than any of these.  Windows of 16, 8 lanes of up to 16k, 16 rows a wave: 88 and 7 us
// (the join) with 256, 76 and 9 with 512, 87 and 11 with 768, 86 and 13 with
// 1024.
constexpr int kFew4Blocks = 2048, kRows4Blocks = 512;
// From this many rows on four waves join a row that may have many splits: 585
// rows of up to 79 splits take 4.7 us, and 8.6 with the 16 waves that a few
// rows of many splits need.
constexpr long kFewRows = 256;

static Shape shape4_of(const gdn_kv_dims& d) {
  return shape_of(d, kFew4Blocks, kRows4Blocks);
}

template <int D, typename T, int RT>
static hipError_t few4(const gdn_kv_dims& d, dim3 grid, const Attend4Args& p,
                       const gdn::LaneTable& tl, hipStream_t st) {
  return d.page_size % 16 == 0
             ? launch(attend4_kernel<D, T, RT, true>, grid, dim3(256), st, p, tl)
             : launch(attend4_kernel<D, T, RT, false>, grid, dim3(256), st, p, tl);
}

template <int D, typename T>
static hipError_t attend4(const gdn_kv_dims& d, const Shape& s,
                          const Attend4Args& p, const gdn::LaneTable& tl,
                          hipStream_t st) {
  const dim3 grid((unsigned)((long)s.items * d.h_kv * s.groups));
  hipError_t e;
  if (!s.few) {
    if constexpr (D < 256) {
      // (128 rows a workgroup: kWide of what the registers hold, see there)
      constexpr int kWaves = kWide<D, T> ? 4 : 8;
      e = s.waves == 8
              ? launch(rows4_kernel<D, T, kWaves, 8 / kWaves>, grid,
                       dim3(64 * kWaves), st, p, tl)
              : launch(rows4_kernel<D, T, 4, 1>, grid, dim3(256), st, p, tl);
    } else {
      e = launch(rows4_kernel<D, T, 4, 1>, grid, dim3(256), st, p, tl);
    }
  } else if constexpr (D < 256) {
    e = s.rt == 2 ? few4<D, T, 2>(d, grid, p, tl, st)
                  : few4<D, T, 1>(d, grid, p, tl, st);
  } else {
    e = few4<D, T, 1>(d, grid, p, tl, st);
  }
  if (e != hipSuccess) return e;
  return (long)d.n_lanes * d.h_kv * s.rows >= kFewRows ? join<D, 4>(d, s, p.at, tl, st)
                                                       : join<D>(d, s, p.at, tl, st);
}

template <typename T>
static hipError_t attend4(const gdn_kv_dims& d, const Shape& s,
                          const Attend4Args& p, const gdn::LaneTable& tl,
                          hipStream_t st) {
  if (d.d == 64) return attend4<64, T>(d, s, p, tl, st);
  if (d.d == 128) return attend4<128, T>(d, s, p, tl, st);
  return attend4<256, T>(d, s, p, tl, st);
}

}  // namespace gdnk

extern "C" size_t gdn_paged_attention_mxfp_workspace_bytes(
    const gdn_kv_dims* dims) {
  if (gdnk::check_kv_dims("gdn_paged_attention_mxfp_workspace_bytes", dims) !=
          GDN_OK ||
      !gdnk::rows_fit(*dims))
    return 0;
  return gdnk::slot_bytes(*dims, gdnk::shape4_of(*dims));
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
  if (!rows_fit(*dims))
    return fail(GDN_EINVAL, "gdn_paged_attention_mxfp: 2^32 rows or more in the cache");
  const size_t need = gdn_paged_attention_mxfp_workspace_bytes(dims);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(GDN_EWORKSPACE, "gdn_paged_attention_mxfp: workspace too small");
  gdn::LaneTable tl;
  int any;
  rc = check_lanes(fn, *dims, t_lane, tl, any);
  if (rc != GDN_OK) return rc;
  if (!any) return GDN_OK;
  const Shape s = shape4_of(*dims);
  Attend4Args p;
  p.at.kv = kv_args(*dims, nullptr, nullptr, page_table, kv_len);
  p.at.q = q;
  p.at.o = o;
  p.at.part_o = (float*)workspace;
  p.at.part_ml = p.at.part_o + (size_t)s.slots * dims->h_kv * s.rows * dims->d;
  p.at.scale = fabsf(scale) * kLog2e;
  p.at.target = s.target;
  p.at.rows = s.rows;
  p.at.groups = s.groups;
  p.flip = !(scale < 0.f) ? 0u : dtype == GDN_BF16 ? 0x80008000u : 0x80000000u;
  p.k4 = {(uint8_t*)k_codes, (uint8_t*)k_scales};
  p.v4 = {(uint8_t*)v_codes, (uint8_t*)v_scales};
  const hipError_t e =
      dtype == GDN_BF16
          ? attend4<uint16_t>(*dims, s, p, tl, (hipStream_t)stream)
          : attend4<float>(*dims, s, p, tl, (hipStream_t)stream);
  return gdn::hip_status(e, "gdn_paged_attention_mxfp launch");
}
