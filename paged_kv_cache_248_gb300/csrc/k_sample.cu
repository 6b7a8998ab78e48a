// k_sample.cu -- tokens drawn from logits, with temperature, top-k, min-p and top-p.
//
// Mathematics.  The candidates of a row in order (larger logit first, of equal ones the lower index) have the
// weights w = exp((x - max) / T).  Every filter keeps a beginning of that order: the first k; those with
// w >= min_p; the shortest with mass >= top_p of what is left.  The token is the first whose cumulative
// weight exceeds u times the kept mass.  Whether a sum of a hundred thousand weights lies above or below
// a border is decided by its last digits, so weights near a border are whole numbers: w 2^S rounded, right to about 2^-40
// of w (weight.cuh), and sums of them exact, in any order.
//
// Work.  A row belongs to a cluster of CTAs, which go through it three times (twice from L2):
//   1. its largest and its least logit;
//   2. how many candidates fall into each of 2048 bins of (max - x) / T, 1/64 of a power of two wide or less, and the sum
//      of their places within it, to 1/32 of it.  That tells the mass up to a bin and the mass behind it to 2e-4 of
//      themselves (ln 2 / 64 / 64 for the places, an eighth of the square of a bin's width for taking the weight of their mean),
//      and so, for each border (the end of top-k and min-p, of top-p, the token), the one or two bins in which it must lie;
//   3. the candidates of those bins are collected, bin by bin, in the cluster's first CTA, and the others' weights summed up
//      between them: exact ones of the first bins, the rest in fp32.
// The first bins are those without which the squares of the others' masses would be more than 2^-8 of the square of the
// kept mass: an fp32 weight is off by 2^-24 (the exponential unit's error, rms, with a mean of -5.25e-8, measured, that is
// given back), so that sums are right to 2^-28 even where all weights of a bin are off the same way (equal logits).
// What was collected (tens to hundreds, where the borders lie in counted bins) is put in order by all CTAs, with exact weights, and the first CTA finds the borders.
// Where one lies so close to a candidate's (2^-25 of the sums, eight times their error) that the fp32 weights could tell them
// wrong, the sums are taken again, exact down to 2^-20 of the largest weight, and the borders found again: a few rows in a
// thousand flat ones, hardly any other.  Weights to be exact wait in a queue of each thread's, so that a warp computes as many
// as it has lanes at a time.  With top-k or min-p nothing behind their end is looked at closely.
// Where more than 2048 candidates lie in the borders' bins, borders are found by bisection of the keys instead, a pass over the
// row each.  Rows of thousands of equal logits come to that (64 rows of 128256: 0.7 ms), and rows with a top-k and no
// min-p whose k-th logit lies behind the counted bins, more than 32 powers of two, 22 temperatures, below the largest.
// Ordinary settings reach that: 64 rows of 32000 (128256) with a top-k of 50 take 19 (29) us at a temperature of 1, 955
// (1383) at 0.3 and 1087 (1834) at 0.2, with 1000 22 (39), 1321 (2326) and 1330 (2358).  A min-p of 2^-31 or more ends the plan before.
//
// Bound: steps, not bytes.  64 rows of 128256 in bf16, four CTAs each, two on most SMs: 43.5 us (2.5 at the HBM copy's rate), in
// clocks of the longest rows: first pass 6000, counts 15000, joining them and the plan 10000, sums 22000, order
// 4000, borders 4000; a pass issues 15 to 25 instructions a logit.  One row of 32000: 13 us, of which the plan takes 2.5, the
// three passes 1.3 each and six cluster barriers 0.6 each.
#include <cooperative_groups.h>

#include "pkv_internal.cuh"
#include "weight.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPerThread = kBins / kThreads;
constexpr float kBinsPerUnit = 64.f;
constexpr float kExactAgain = 20.f;  // weights down to 2^-20 of the largest are exact where sums are taken again
constexpr float kRest = 1.f / 256.f;  // squares of the bins' masses that fp32 weights may leave, of the kept mass's
constexpr int kCollect = 2048;
// Candidates whose borders a warp finds alone: of 32, 64, 128, 256 at most 64 rows of 128256 take 44.1, 43.8, 43.5, 44.2 us, 256 of 32000
// 43.0, 42.1, 41.6, 41.9; one row, which has a few, 12.9, and 15.2 where the CTA always does.
constexpr int kFew = 128;
constexpr int kQueue = 16;  // places of a thread's queue, eight of which a piece may fill

struct Params {
  const void* logits;
  int64_t stride;
  const float *temperature, *top_p, *min_p, *uniform;
  const int32_t* top_k;
  int32_t* tokens;
  float* logprobs;
  uint32_t* err;
  int32_t vocab, shift;
};

// What the counts tell: up to three disjoint intervals of bins that are collected.
struct Plan {
  int32_t begin[3], end[3];  // bins [begin, end], kBins where there are fewer
  int32_t last;              // bins behind it are ignored
  int32_t exact;             // weights of the bins before are exact
  int32_t rank[3];           // candidate number e of the list, in interval j, is number rank[j] + e of the row
};

struct Shared {
  uint32_t bins[kBins], places[kBins];  // of this CTA: candidates, and the sum of their places in the bin
  uint32_t all[kBins];                  // of the row: candidates, and the mean of their places
  union {
    float mean[kBins];
    int32_t base[kBins];  // (after the plan) where the list has a collected bin's candidates
  };
  uint32_t cursor[kBins];  // (first CTA) of a bin's candidates, those that have a place in the list
  uint64_t list[kCollect], weights[kCollect];  // (first CTA) keys, at last in order, and their weights
  union {
    float queue[kQueue][kThreads];
    struct {  // after the queues
      uint64_t unsorted[kCollect], sorted[kCollect];  // (`sorted`: first CTA)
    };
  };
  uint64_t table[256];
  float largest[16], least[16];  // of each CTA's candidates
  unsigned long long segment[3];  // masses of what is not collected: before the intervals, and behind the first ones
  unsigned long long warp_u64[kWarps];
  float warp_mass[kWarps], warp_low[kWarps];
  uint32_t warp_n[kWarps];
  int32_t found[6], counts[6];  // (of the plan)
  float warp_sq[kWarps], bound[4];
  uint32_t collected, best;  // (first CTA) of the list; the first of the largest logits
  uint32_t taken;            // candidates that this CTA collected (in `weights`)
  int32_t unsure;            // (first CTA) the borders need exact sums
  Plan plan;
  unsigned long long sum[2], low, high;  // of a pass of the bisection
};

// Larger logits have smaller keys; the index in the lower half.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 as 0)
  return ~(u & 0x80000000u ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float x, int i) { return static_cast<uint64_t>(order_of(x)) << 32 | static_cast<uint32_t>(i); }
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t up = ~static_cast<uint32_t>(key >> 32);
  return __uint_as_float(up & 0x80000000u ? up & 0x7fffffffu : ~up);
}
__device__ __forceinline__ bool candidate(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// A piece of a row: eight logits, 16 or 32 bytes.
constexpr int kPiece = 8;
template <typename T>
struct Piece {
  uint4 v[kPiece * sizeof(T) / 16];
};

// The piece that begins at logit i0; what does not belong to the row is NaN, no candidate.
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* p, int i0, int vocab) {
  Piece<T> piece;
  constexpr int kParts = sizeof(piece) / 16;
  if (i0 >= 0 && i0 + kPiece <= vocab) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) piece.v[k] = __ldg(reinterpret_cast<const uint4*>(p + i0) + k);
    return piece;
  }
#pragma unroll
  for (int k = 0; k < kParts; ++k) piece.v[k] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
  if (i0 >= vocab) return piece;
  uint32_t* w = reinterpret_cast<uint32_t*>(piece.v);
#pragma unroll
  for (int e = 0; e < kPiece; ++e) {
    if (i0 + e < 0 || i0 + e >= vocab) continue;
    const uint32_t x = __float_as_uint(Elem<T>::to_f32(p[i0 + e]));
    if constexpr (sizeof(T) == 4) w[e] = x;
    else w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | x : (w[e / 2] & 0xffff0000u) | x >> 16;
  }
  return piece;
}

// Calls f(piece, i) with this thread's pieces of the row (`first`, first + step, ...), whose logits begin at number i.  All threads of
// a CTA call it equally often.  The next pieces, 48 (32) bytes of them, are on their way while one is worked on.
template <typename T, typename F>
__device__ __forceinline__ void each_raw(const Params& P, int64_t row, int first, int step, F&& f) {
  const T* p = static_cast<const T*>(P.logits) + row * P.stride;
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));  // piece 0 begins so much before
  const int end = skew + P.vocab;
  int i0 = first * kPiece - skew;
  const int hop = step * kPiece;
  constexpr int kAhead = sizeof(T) == 4 ? 1 : 3;
  Piece<T> ring[kAhead + 1];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) ring[k] = load_piece<T>(p, i0 + k * hop, P.vocab);
#pragma unroll 1
  for (int v = first - static_cast<int>(threadIdx.x); v * kPiece < end; v += step, i0 += hop) {
    ring[kAhead] = load_piece<T>(p, i0 + kAhead * hop, P.vocab);
    f(ring[0], i0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ring[k] = ring[k + 1];
  }
}
template <typename T>
__device__ __forceinline__ void unpack_piece(const Piece<T>& piece, float (&x)[kPiece]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(piece.v);
#pragma unroll
  for (int e = 0; e < kPiece; ++e)
    x[e] = __uint_as_float(sizeof(T) == 4 ? w[e] : e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
}
// The largest logit of a piece (NaN is passed over).
template <typename T>
__device__ __forceinline__ float piece_largest(const Piece<T>& piece) {
  if constexpr (sizeof(T) == 4) {
    const float* x = reinterpret_cast<const float*>(piece.v);
    return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  } else {
    const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(piece.v);
    const __nv_bfloat162 y = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
    return fmaxf(__low2float(y), __high2float(y));
  }
}
// The same with their logits x[].
template <typename T, typename F>
__device__ __forceinline__ void each_piece(const Params& P, int64_t row, int first, int step, F&& f) {
  each_raw<T>(P, row, first, step, [&](const Piece<T>& raw, int i0) {
    float x[kPiece];
    unpack_piece<T>(raw, x);
    f(x, i0);
  });
}
// f(x, i) for each of them.
template <typename T, typename F>
__device__ __forceinline__ void each(const Params& P, int64_t row, int first, int step, F&& f) {
  each_piece<T>(P, row, first, step, [&](const float (&x)[kPiece], int i0) {
#pragma unroll
    for (int e = 0; e < kPiece; ++e) f(x[e], i0 + e);
  });
}

// Adds to a word of shared memory where |y| < end.
__device__ __forceinline__ void add_below(float y, float end, uint32_t addr, uint32_t x) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .f32 a;\n\tabs.f32 a, %0;\n\tsetp.lt.f32 p, a, %1;\n\t@p red.shared.add.u32 [%2], %3;\n\t}" ::"f"(y), "f"(end),
      "r"(addr), "r"(x)
      : "memory");
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ uint64_t warp_min(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = min(x, static_cast<uint64_t>(__shfl_xor_sync(0xffffffffu, x, d)));
  return x;
}
// Inclusive sums over the block's threads; *all: the sum of all.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, Shared& s, uint64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s.warp_u64[warp] = x;
  __syncthreads();
  uint64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const uint64_t y = s.warp_u64[w];
    if (w < warp) before += y;
    sum += y;
  }
  __syncthreads();
  *all = sum;
  return x + before;
}
__device__ __forceinline__ uint64_t block_sum(uint64_t x, Shared& s) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) s.warp_u64[threadIdx.x >> 5] = x;
  __syncthreads();
  uint64_t sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += s.warp_u64[w];
  __syncthreads();
  return sum;
}
__device__ __forceinline__ uint64_t block_min(uint64_t x, Shared& s) {
  x = warp_min(x);
  if ((threadIdx.x & 31) == 0) s.warp_u64[threadIdx.x >> 5] = x;
  __syncthreads();
  uint64_t least = s.warp_u64[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) least = min(least, static_cast<uint64_t>(s.warp_u64[w]));
  __syncthreads();
  return least;
}

// Settings of a row.
struct Row {
  float temperature, top_p, min_p, u;
  int32_t top_k;
};

// The borders' bins, from the row's counts (every CTA makes the same plan).  The last bin's candidates are not
// counted: there are `rest` of their weights, 2^-32 each, at most.
__device__ __forceinline__ void make_plan(Shared& s, const Row& r, float per_unit, float rest) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = threadIdx.x * kPerThread;
  static_assert(kPerThread == 4, "a thread's bins are a vector");
  const uint4 x = *reinterpret_cast<const uint4*>(s.all + b0);
  const float4 y = *reinterpret_cast<const float4*>(s.mean + b0);
  uint32_t n[4] = {x.x, x.y, x.z, x.w};
  const float mean[4] = {y.x, y.y, y.z, y.w};
  // candidates of these bins and up to each, and the mass up to each
  const uint32_t here[4] = {n[0], n[1], n[2], n[3]};
  float mass[4], sq[4], behind[4];  // (and the squares of the bins' masses; the mass behind each)
  uint32_t counted = 0;
  float weighed = 0.f, squares = 0.f;
  const float unit = 1.f / per_unit;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float m = here[k] * ex2_approx(-(static_cast<float>(b0 + k) + mean[k]) * unit);
    behind[k] = m;
    weighed += m;
    squares = fmaf(m, m, squares);
    counted += here[k];
    n[k] = counted;
    mass[k] = weighed;
    sq[k] = squares;
  }
  {
    const float m3 = behind[3], m2 = behind[2], m1 = behind[1];
    behind[3] = 0.f;
    behind[2] = m3;
    behind[1] = m2 + m3;
    behind[0] = m1 + behind[1];
  }
  uint32_t in = counted;
  float im = weighed, is = squares, ib = weighed;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, in, d);
    const float z = __shfl_up_sync(0xffffffffu, im, d), x = __shfl_up_sync(0xffffffffu, is, d), v = __shfl_down_sync(0xffffffffu, ib, d);
    if (lane >= d) {
      in += y;
      im += z;
      is += x;
    }
    if (lane + d < 32) ib += v;
  }
  if (lane == 31) {
    s.warp_n[warp] = in;
    s.warp_mass[warp] = im;
    s.warp_sq[warp] = is;
  }
  if (threadIdx.x < 6) s.found[threadIdx.x] = kBins - 1;
  __syncthreads();
  // (the warps' sums: lane w has those up to warp w)
  uint32_t wn = lane < kWarps ? s.warp_n[lane] : 0;
  float wm = lane < kWarps ? s.warp_mass[lane] : 0.f, ws = lane < kWarps ? s.warp_sq[lane] : 0.f, wb = wm;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, wn, d);
    const float z = __shfl_up_sync(0xffffffffu, wm, d), x = __shfl_up_sync(0xffffffffu, ws, d), v = __shfl_down_sync(0xffffffffu, wb, d);
    if (lane >= d) {
      wn += y;
      wm += z;
      ws += x;
    }
    if (lane + d < 32) wb += v;
  }
  const float all = __shfl_sync(0xffffffffu, wm, kWarps - 1), all_sq = __shfl_sync(0xffffffffu, ws, kWarps - 1);
  uint32_t bn = __shfl_sync(0xffffffffu, wn, max(warp - 1, 0));
  float bm = __shfl_sync(0xffffffffu, wm, max(warp - 1, 0)), bs = __shfl_sync(0xffffffffu, ws, max(warp - 1, 0));
  float bb = __shfl_sync(0xffffffffu, wb, warp + 1);  // (nothing in lane kWarps)
  if (warp == 0) {
    bn = 0;
    bm = bs = 0.f;
  }
  bn += in - counted;
  bm += im - weighed;
  bs += is - squares;
  const float next = __shfl_down_sync(0xffffffffu, ib, 1);
  bb += lane < 31 ? next : 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    n[k] += bn;
    mass[k] += bm;
    sq[k] += bs;
    behind[k] += bb;
  }
  // the masses above are off by a part of 2e-4 at most, and by what lies behind the last bin
  constexpr float kLow = 0.9998f, kHigh = 1.0002f;
  const auto first_of = [&](int at, bool y0, bool y1, bool y2, bool y3) {  // the first bin of which it holds, and of all behind
    const int mine = __reduce_min_sync(0xffffffffu, y3 ? b0 + (y0 ? 0 : y1 ? 1 : y2 ? 2 : 3) : kBins - 1);
    if (lane == 0 && mine < kBins - 1) atomicMin(&s.found[at], mine);
  };
  const bool cut_k = r.top_k > 0, cut_m = r.min_p > 0.f;  // (a top-k of all and more ends in the last bin)
  if (cut_k) {
    const uint32_t k = static_cast<uint32_t>(r.top_k);
    const int at = n[0] >= k ? 0 : n[1] >= k ? 1 : n[2] >= k ? 2 : 3;
    if (bn < k && n[3] >= k) s.found[0] = b0 + at;
    __syncthreads();
  }
  int a1 = kBins, e1 = kBins - 1;  // the end of top-k and min-p
  if (cut_k) a1 = e1 = s.found[0];
  if (cut_m) {
    const int at = static_cast<int>(fminf(-log2f(r.min_p) * per_unit, kBins - 1.f));
    a1 = min(a1, max(at - 1, 0));
    e1 = min(e1, min(at + 1, kBins - 1));
  }
  const bool cut1 = cut_k || cut_m;
  // the mass up to there: bounds
  if (cut1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (b0 + k == a1 - 1) {
        s.bound[0] = mass[k];
        s.bound[2] = behind[k];
      }
      if (b0 + k == e1) {
        s.bound[1] = sq[k];
        s.bound[3] = behind[k];
      }
    }
    if (threadIdx.x == 0 && a1 == 0) s.bound[0] = 0.f, s.bound[2] = all;
    __syncthreads();
  }
  const float z_lo = (cut1 ? s.bound[0] : all) * kLow;
  {  // the first bins, until the rest's squares are 2^-8 of the kept mass's
    const float x = (cut1 ? s.bound[1] : all_sq) - z_lo * z_lo * kRest;
    first_of(5, sq[0] > x, sq[1] > x, sq[2] > x, sq[3] > x);
  }
  // A share f of the kept mass is passed where f S < (1 - f) M, of the mass M up to a bin and S of the kept behind it: as tight
  // near the end, where S is small and its bins are full, as at the beginning.  The first bin where that can be (f = lo), and
  // where it must be (f = hi).
  const float less = cut1 ? s.bound[2] * kHigh : 0.f, least = cut1 ? s.bound[3] * kLow : 0.f;
  const auto borders = [&](int at, float lo, float hi) {
    bool can[4], must[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      can[k] = lo * (behind[k] * kLow - less) < (1.f - lo) * (mass[k] * kHigh);
      must[k] = hi * (behind[k] * kHigh - least + rest) < (1.f - hi) * (mass[k] * kLow);
    }
    first_of(at, can[0], can[1], can[2], can[3]);
    first_of(at + 1, must[0], must[1], must[2], must[3]);
  };
  // the end of top-p
  int a2 = kBins, e2 = e1;
  const bool cut_p = r.top_p < 1.f;
  float kept_lo = 1.f, kept_hi = 1.f;  // top-p's share with what its last candidate adds
  if (cut_p) {
    borders(1, r.top_p, r.top_p);
    __syncthreads();
    a2 = min(s.found[1], e1);
    e2 = min(s.found[2], e1);
    kept_lo = r.top_p * 0.9999998f;
    kept_hi = fminf(1.f, r.top_p * 1.0000002f + kHigh * ex2_approx(-static_cast<float>(a2) * unit) / z_lo);
  }
  borders(3, r.u * kept_lo, r.u * kept_hi);
  __syncthreads();
  // three windows in order of their beginnings, joined where they meet (kBins: none)
  const int a3 = min(s.found[3], e2), e3 = min(s.found[4], e2), exact = s.found[5] + 1;
  int a[3] = {a3, cut_p ? a2 : kBins, cut1 ? a1 : kBins}, e[3] = {max(a3, e3), max(a2, e2), max(a1, e1)};
  const auto swap = [&](int x, int y, bool really) {
    const int u = really ? a[y] : a[x], v = really ? e[y] : e[x];
    a[y] = really ? a[x] : a[y], e[y] = really ? e[x] : e[y];
    a[x] = u, e[x] = v;
  };
  swap(0, 1, a[1] < a[0]);
  swap(1, 2, a[2] < a[1]);
  swap(0, 1, a[1] < a[0]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // (what a window takes up is moved to the end)
#pragma unroll
    for (int k = 0; k < 2 - i; ++k) {
      const bool meet = a[i + 1] < kBins && a[i + 1] <= e[i] + 1;
      e[i] = meet ? max(e[i], e[i + 1]) : e[i];
      a[i + 1] = meet ? kBins : a[i + 1];
      if (i == 0) swap(1, 2, a[2] < a[1]);
    }
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) e[j] = a[j] < kBins ? e[j] : kBins;
  // candidates before an interval, and up to its end
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      if (a[j] == b0 + k) s.counts[j] = static_cast<int32_t>(n[k] - here[k]);
      if (e[j] == b0 + k) s.counts[3 + j] = static_cast<int32_t>(n[k]);
    }
  }
  __syncthreads();
  int rank[3], collected = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    rank[j] = s.counts[j] - collected;
    collected += a[j] < kBins ? s.counts[3 + j] - s.counts[j] : 0;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = b0 + k;
    s.base[b] = static_cast<int32_t>(n[k] - here[k]) - (b >= a[2] ? rank[2] : b >= a[1] ? rank[1] : rank[0]);
  }
  if (threadIdx.x == 0) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      s.plan.begin[j] = a[j];
      s.plan.end[j] = e[j];
      s.plan.rank[j] = rank[j];
    }
    s.plan.last = cut1 ? e1 : kBins - 1;
    s.plan.exact = exact;
  }
  __syncthreads();
}

// The bin of a place.
__device__ __forceinline__ int bin_of(float y) {
  return __float_as_uint(__fadd_rd(fminf(y, (kBins - 1) * 2048.f), 8388608.f)) >> 11 & (kBins - 1);
}

// Sorts the n keys of `unsorted`, which are in order of their bins, into the first CTA's `sorted`, with their weights: each
// key's place is the number of smaller ones of its bin behind the bin's first, which the lanes of a group count
// together.  Every CTA of the cluster takes a share of them.
template <int kCtas>
__device__ __forceinline__ void rank_share(Shared& s, Shared* head, const Weight& w, float per_place, int n, int rank) {
  const int e0 = n * rank / kCtas, e1 = n * (rank + 1) / kCtas;
  int group = 1;
  while (group < 32 && (e1 - e0) * group * 2 <= kThreads) group <<= 1;
  const int at = threadIdx.x & (group - 1);
#pragma unroll 1
  for (int first = e0; first < e1; first += kThreads / group) {
    const int e = first + static_cast<int>(threadIdx.x) / group;
    const uint64_t mine = s.unsorted[min(e, e1 - 1)];
    const float x = logit_of(mine);
    // (the last bin's are not counted; bounds, so that logits which are written meanwhile cannot lead out of the list)
    const int bin = bin_of((w.top - x) * per_place), begin = min(max(s.base[bin], 0), n - 1);
    const int end = bin == kBins - 1 ? n : min(begin + static_cast<int>(min(s.all[bin], 1u << 20)), n);
    int place = 0;
#pragma unroll 4
    for (int i = begin + at; i < end; i += group) place += s.unsorted[i] < mine;
    __syncwarp();
#pragma unroll 1
    for (int d = group >> 1; d; d >>= 1) place += __shfl_xor_sync(0xffffffffu, place, d);
    if (e < e1 && at == 0) {
      const int to = min(begin + place, n - 1);
      head->sorted[to] = mine;
      head->weights[to] = w.of(x, s.table);
    }
  }
}

// The same of many keys, by the first CTA.
__device__ __forceinline__ void sort_many(Shared& s, const Weight& w, int n) {
  int size = kThreads;
  while (size < n) size <<= 1;
  for (int i = threadIdx.x; i < size; i += kThreads) s.sorted[i] = i < n ? s.unsorted[i] : ~uint64_t(0);
  __syncthreads();
#pragma unroll 1
  for (int k = 2; k <= size; k <<= 1) {
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
#pragma unroll 1
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;  // bit j of a is 0
        const uint64_t x = s.sorted[a], y = s.sorted[b];
        if ((x > y) == ((a & k) == 0)) {
          s.sorted[a] = y;
          s.sorted[b] = x;
        }
      }
      // (pairs up to 32 apart stay within a warp's 64 places)
      if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
      else __syncwarp();
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kThreads) s.weights[i] = w.of(logit_of(s.sorted[i]), s.table);
}

// The same of at most 32 keys of `list`, in place, by a warp of the first CTA.
__device__ __forceinline__ void rank_few(Shared& s, const Weight& w, int n) {
  const int lane = threadIdx.x & 31;
  const uint64_t mine = lane < n ? s.list[lane] : ~uint64_t(0);
  int place = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) place += __shfl_sync(0xffffffffu, mine, i) < mine;
  __syncwarp();
  if (lane < n) {
    s.list[place] = mine;
    s.weights[place] = w.of(logit_of(mine), s.table);
  }
  __syncwarp();
}

// Sums up to each thread and over all, a sum, a minimum, a vote: of a warp, or of all threads of the CTA.
template <bool kWarp>
struct Team {
  Shared& s;
  __device__ __forceinline__ uint64_t scan(uint64_t x, uint64_t* all) {
    if constexpr (!kWarp) return block_scan(x, s, all);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    *all = __shfl_sync(0xffffffffu, x, 31);
    return x;
  }
  __device__ __forceinline__ uint64_t sum(uint64_t x) { return kWarp ? warp_sum(x) : block_sum(x, s); }
  __device__ __forceinline__ uint64_t least(uint64_t x) { return kWarp ? warp_min(x) : block_min(x, s); }
  __device__ __forceinline__ bool any(bool x) { return kWarp ? __any_sync(0xffffffffu, x) != 0 : __syncthreads_or(x) != 0; }
};

// The token out of the n collected candidates, which are sorted (the first CTA, or its first warp): 0.  1: with `exact` sums between them it
// could be another.  2: it is not among them.
template <bool kWarp>
__device__ __forceinline__ int finish(const Params& P, Shared& s, const Row& r, const Weight& w, float per_place, int64_t row, int n,
                                    bool exact) {
  const Plan p = s.plan;
  const uint64_t least_w = r.min_p > 0.f ? w.part_up(r.min_p) : 0;
  const uint32_t most = r.top_k > 0 ? static_cast<uint32_t>(r.top_k) : 0xffffffffu;
  constexpr int kTeam = kWarp ? 32 : kThreads;
  Team<kWarp> team{s};
  const int per = (n + kTeam - 1) / kTeam, e0 = threadIdx.x * per, e1 = min(e0 + per, n);
  // the mass before the intervals, of what is not collected
  const uint64_t seg0 = s.segment[0], seg1 = seg0 + s.segment[1], segs = seg1 + s.segment[2], seg2 = segs;
  // a candidate's interval, from its bin
  const auto interval = [&](int e) {
    const int b = bin_of((w.top - logit_of(s.list[e])) * per_place);
    return (b >= p.begin[1]) + (b >= p.begin[2]);
  };
  const auto rank_of = [&](int e, int j) { return static_cast<uint32_t>((j == 0 ? p.rank[0] : j == 1 ? p.rank[1] : p.rank[2]) + e); };
  uint64_t mine = 0, kept = 0, all;
#pragma unroll 1
  for (int e = e0; e < e1; ++e) {
    const uint64_t m = s.weights[e];
    mine += m;
    if (m >= least_w && rank_of(e, interval(e)) < most) kept += m;
  }
  const uint64_t first = team.scan(mine, &all) - mine;  // of this thread's part
  const uint64_t z1 = team.sum(kept) + segs;
  const uint64_t off = exact || segs == 0 ? 0 : z1 >> 25;  // how far sums may be off
  bool unsure = false;
  // What is kept after top-p, and the token, of this thread's part.
  const uint64_t share = fraction64(r.top_p), p_hi = __umul64hi(z1, share), p_lo = z1 * share;
  uint64_t z2 = z1, token = ~uint64_t(0), target = 0;
#pragma unroll 1
  for (int pass = r.top_p < 1.f ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) target = part_of(z2, r.u);
    uint64_t at = first, top = 0;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      const int j = interval(e);
      const uint64_t m = s.weights[e], upto = (j == 0 ? seg0 : j == 1 ? seg1 : seg2) + at;
      at += m;
      if (pass == 1) {
        unsure |= upto + m <= target + off && upto + m + off >= target && off > 0;
        if (upto + m > target) token = min(token, static_cast<uint64_t>(e));
      } else {
        unsure |= upto <= p_hi + off && upto + off >= p_hi && off > 0;
        const uint32_t rank = rank_of(e, j);
        if (rank < most && m >= least_w && (rank == 0 || upto < p_hi || (upto == p_hi && p_lo != 0))) top = upto + m;
      }
    }
    const uint64_t least = team.least(pass == 1 ? token : ~top);
    if (pass == 1) token = least;
    else z2 = ~least;
  }
  if (team.any(unsure)) return 1;
  if (token == ~uint64_t(0)) return 2;
  if (threadIdx.x == 0) {
    const int e = static_cast<int>(token);
    const uint64_t key = s.list[e];
    P.tokens[row] = static_cast<int32_t>(key & 0xffffffffu);
    if (P.logprobs) P.logprobs[row] = w.log_share(logit_of(key), r.temperature, s.weights[e], z2);
  }
  return 0;
}

// ------------------------------------------------------------------ bisection
// Of the candidates with keys in (from, to]: how many there are and their mass; of those behind `to` and up to `end`: the
// least and the largest key.  (All CTAs of the cluster; the same answer in each.)
template <typename T, int kCtas>
__device__ __noinline__ void look(const Params& P, Shared& s, const Weight& w, int64_t row, int rank, uint64_t to, uint64_t end,
                                  uint64_t* count, uint64_t* mass, uint64_t* least, uint64_t* most) {
  cg::cluster_group cluster = cg::this_cluster();
  uint64_t n = 0, m = 0, lo = ~uint64_t(0), hi = 0;
  each<T>(P, row, rank * kThreads + threadIdx.x, kCtas * kThreads, [&](float x, int i) {
    if (!candidate(x)) return;
    const uint64_t key = key_of(x, i);
    if (key <= to) {
      ++n;
      m += w.of(x, s.table);
    } else if (key <= end) {
      lo = min(lo, key);
      hi = max(hi, key);
    }
  });
  if (threadIdx.x == 0) {
    s.sum[0] = s.sum[1] = s.high = 0;
    s.low = ~0ull;
  }
  __syncthreads();
  n = warp_sum(n);
  m = warp_sum(m);
  lo = warp_min(lo);
  hi = ~warp_min(~hi);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&s.sum[0], static_cast<unsigned long long>(n));
    atomicAdd(&s.sum[1], static_cast<unsigned long long>(m));
    atomicMin(&s.low, static_cast<unsigned long long>(lo));
    atomicMax(&s.high, static_cast<unsigned long long>(hi));
  }
  cluster.sync();
  *count = *mass = *most = 0;
  *least = ~uint64_t(0);
  for (int c = 0; c < kCtas; ++c) {
    const Shared* o = cluster.map_shared_rank(&s, c);
    *count += o->sum[0];
    *mass += o->sum[1];
    *least = min(*least, static_cast<uint64_t>(o->low));
    *most = max(*most, static_cast<uint64_t>(o->high));
  }
  cluster.sync();
}

// The least key of a candidate up to which enough(count, mass) holds; one up to `end` has it.
template <typename T, int kCtas, typename Enough>
__device__ __forceinline__ uint64_t bisect(const Params& P, Shared& s, const Weight& w, int64_t row, int rank, uint64_t end,
                                           Enough&& enough) {
  uint64_t count, mass, lo, hi;  // the answer is one of the candidates from lo to hi
  look<T, kCtas>(P, s, w, row, rank, 0, end, &count, &mass, &lo, &hi);
  if (enough(count, mass)) return 0;  // (key 0 is no finite logit's)
  while (lo < hi) {
    const uint64_t mid = lo + (hi - lo) / 2;
    uint64_t next_lo, next_hi;
    look<T, kCtas>(P, s, w, row, rank, mid, hi, &count, &mass, &next_lo, &next_hi);
    if (enough(count, mass)) {
      hi = mid;
    } else {
      lo = next_lo;
      hi = next_hi;
    }
  }
  return hi;
}

template <typename T, int kCtas>
__device__ __noinline__ void by_bisection(const Params& P, Shared& s, const Row& r, const Weight& w, int64_t row, int rank) {
  const uint64_t all = ~uint64_t(0);
  uint64_t end = all, count, mass, x, y;
  look<T, kCtas>(P, s, w, row, rank, all, all, &count, &mass, &x, &y);
  if (r.top_k > 0 && static_cast<uint64_t>(r.top_k) < count)
    end = bisect<T, kCtas>(P, s, w, row, rank, all, [&](uint64_t n, uint64_t) { return n >= static_cast<uint64_t>(r.top_k); });
  if (r.min_p > 0.f) {
    // kept are the keys up to the last whose weight is enough: weights fall with the keys
    const uint64_t least_w = w.part_up(r.min_p);
    uint64_t lo = 0, hi = 0xffffffffu;  // of the order: the last one with enough
    while (lo < hi) {
      const uint64_t mid = lo + (hi - lo + 1) / 2;
      const float logit = logit_of(mid << 32);
      // (orders before the largest logit's are no candidates')
      if (mid <= order_of(w.top) || (candidate(logit) && w.of(logit, s.table) >= least_w)) lo = mid;
      else hi = mid - 1;
    }
    end = min(end, lo << 32 | 0xffffffffu);
  }
  look<T, kCtas>(P, s, w, row, rank, end, end, &count, &mass, &x, &y);
  if (r.top_p < 1.f) {
    const uint64_t want = part_of_up(mass, r.top_p);
    end = bisect<T, kCtas>(P, s, w, row, rank, end, [&](uint64_t n, uint64_t m) { return n >= 1 && m >= want; });
    look<T, kCtas>(P, s, w, row, rank, end, end, &count, &mass, &x, &y);
  }
  const uint64_t target = part_of(mass, r.u);
  const uint64_t key = bisect<T, kCtas>(P, s, w, row, rank, end, [&](uint64_t, uint64_t m) { return m > target; });
  if (rank == 0 && threadIdx.x == 0) {
    P.tokens[row] = static_cast<int32_t>(key & 0xffffffffu);
    if (P.logprobs) P.logprobs[row] = w.log_share(logit_of(key), r.temperature, w.of(logit_of(key), s.table), mass);
  }
}

// ------------------------------------------------------------------ kernel
template <typename T, int kCtas>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 2) sample_kernel(const Params P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCtas == 1 ? 0 : static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / kCtas;
  const int first = rank * kThreads + threadIdx.x, step = kCtas * kThreads;
  if (threadIdx.x < 256) s.table[threadIdx.x] = kPowers.v[threadIdx.x];
  static_assert(kBins == 4 * kThreads, "a vector of bins a thread");
  reinterpret_cast<uint4*>(s.bins)[threadIdx.x] = reinterpret_cast<uint4*>(s.places)[threadIdx.x] =
      reinterpret_cast<uint4*>(s.cursor)[threadIdx.x] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 3) s.segment[threadIdx.x] = 0;
  if (threadIdx.x == 4) s.collected = s.taken = 0;
  if (threadIdx.x == 5) s.best = 0x7fffffffu;
  if constexpr (kCtas > 1) cluster.barrier_arrive();
  grid_dep_wait();
  grid_dep_launch();
  Row r;
  r.temperature = P.temperature ? __ldg(P.temperature + row) : 1.f;
  r.top_p = P.top_p ? __ldg(P.top_p + row) : 1.f;
  r.min_p = P.min_p ? __ldg(P.min_p + row) : 0.f;
  r.top_k = P.top_k ? __ldg(P.top_k + row) : 0;
  r.u = __ldg(P.uniform + row);
  // The largest logit and the least, which may be infinite: -inf makes the bins the coarsest, which they are for most rows;
  // of a row with an infinity above its candidates the largest one is looked for again.
  float top, low;
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    top = -INFINITY, low = INFINITY;
    if (again) {
      each<T>(P, row, first, step, [&](float x, int) {
        const bool is_one = candidate(x);
        top = fmaxf(top, is_one ? x : -INFINITY);
        low = fminf(low, is_one ? x : INFINITY);
      });
    } else if constexpr (sizeof(T) == 4) {
      each<T>(P, row, first, step, [&](float x, int) {  // (NaN is passed over)
        top = fmaxf(top, x);
        low = fminf(low, x);
      });
    } else {
      __nv_bfloat162 hi = __float2bfloat162_rn(-INFINITY), lo = __float2bfloat162_rn(INFINITY);
      each_raw<T>(P, row, first, step, [&](const Piece<T>& raw, int) {
        const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(raw.v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi = __hmax2(hi, x[e]);
          lo = __hmin2(lo, x[e]);
        }
      });
      top = fmaxf(__low2float(hi), __high2float(hi));
      low = fminf(__low2float(lo), __high2float(lo));
    }
    const uint32_t a = __reduce_min_sync(0xffffffffu, order_of(top)), b = __reduce_max_sync(0xffffffffu, order_of(low));
    if ((threadIdx.x & 31) == 0) {
      s.warp_mass[threadIdx.x >> 5] = logit_of(static_cast<uint64_t>(a) << 32);
      s.warp_low[threadIdx.x >> 5] = logit_of(static_cast<uint64_t>(b) << 32);
    }
    __syncthreads();
    // (a CTA's shared memory is there once the CTA runs, which its arrival tells; one row of 32000, 8 CTAs: no difference)
    if constexpr (kCtas > 1) {
      if (!again) cluster.barrier_wait();
    }
    if (threadIdx.x < kCtas) {
      float x = -INFINITY, y = INFINITY;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        x = fmaxf(x, s.warp_mass[v]);
        y = fminf(y, s.warp_low[v]);
      }
      Shared* o = cluster.map_shared_rank(&s, threadIdx.x);
      o->largest[rank] = x;
      o->least[rank] = y;
    }
    cluster.sync();
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      top = fmaxf(c == 0 ? -INFINITY : top, s.largest[c]);
      low = fminf(c == 0 ? INFINITY : low, s.least[c]);
    }
    if (top != INFINITY) break;
    cluster.sync();
  }
  const bool wrong = !(r.temperature >= 0.f && r.temperature < INFINITY) || !(r.u >= 0.f && r.u < 1.f) || !(r.top_p >= 0.f) ||
                     !(r.min_p <= 1.f);
  if (wrong || top == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      if (wrong) flag_error(P.err, kErrSetting);
      P.tokens[row] = -1;
      if (P.logprobs) P.logprobs[row] = -INFINITY;
    }
    return;
  }
  Shared* head = cluster.map_shared_rank(&s, 0);
  if (r.temperature == 0.f) {  // the first of the largest
    uint32_t at = 0x7fffffffu;
    each<T>(P, row, first, step, [&](float x, int i) { at = x == top ? min(at, static_cast<uint32_t>(i)) : at; });
    at = __reduce_min_sync(0xffffffffu, at);
    if ((threadIdx.x & 31) == 0) atomicMin(&head->best, at);
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
      P.tokens[row] = static_cast<int32_t>(s.best);
      if (P.logprobs) P.logprobs[row] = 0.f;
    }
    return;
  }
  const Weight w(top, r.temperature, P.shift);
  // bins a power of two of the weights: 64, or as many as let the row's candidates have all but the last one
  const float range = fmaxf((top - low) * w.ch, 1e-6f);
  const float per_unit = fmaxf(kBinsPerUnit, (kBins - 2.f) / range);
  // A place in the bins in units of 1/2048, behind the binary point of 2^23: bin and place are its bits.
  const float per_place = fminf(w.ch * per_unit, 1e30f) * 2048.f;
  constexpr float kEnd = (kBins - 1) * 2048.f;
  // How many fall into each bin, and where, to 1/32 of it: both in one word while there are few (upper 14 bits and lower 18), two
  // arrays of them in turn; a thread keeps the sums of four bins.
  {
    static_assert(kPerThread == 4, "a thread's bins are a vector");
    constexpr int kPieces = 2;
    static_assert(kPieces * kPiece * kThreads < (1 << 14) && 31 * kPieces * kPiece * kThreads < (1 << 18), "the fields of a word");
    uint32_t into = smem_u32(s.bins);
    const float per_part = per_place * (1.f / 64.f);
    uint32_t n[4] = {0, 0, 0, 0}, place[4] = {0, 0, 0, 0};
    int pieces = 0;
    const auto take_over = [&]() {
      uint32_t* of = into == smem_u32(s.bins) ? s.bins : s.places;
      const uint4 x = reinterpret_cast<const uint4*>(of)[threadIdx.x];
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};
      reinterpret_cast<uint4*>(of)[threadIdx.x] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        n[k] += y[k] >> 18;
        place[k] += y[k] & 0x3ffffu;
      }
    };
    each_piece<T>(P, row, first, step, [&](const float (&x)[kPiece], int) {
#pragma unroll
      for (int e = 0; e < kPiece; ++e) {
        const float y = (top - x[e]) * per_part;
        const uint32_t at = __float_as_uint(__fadd_rd(y, 8388608.f));
        // (not the last bin's, nor what is no candidate)
        add_below(y, kEnd / 64.f, into + ((at & 32u * (kBins - 1)) >> 3), (at & 31u) | 0x40000u);
      }
      if (++pieces == kPieces) {
        pieces = 0;
        __syncthreads();
        take_over();
        into ^= smem_u32(s.bins) ^ smem_u32(s.places);
      }
    });
    __syncthreads();
    take_over();
    reinterpret_cast<uint4*>(s.bins)[threadIdx.x] = make_uint4(n[0], n[1], n[2], n[3]);
    reinterpret_cast<uint4*>(s.places)[threadIdx.x] = make_uint4(place[0], place[1], place[2], place[3]);
  }
  cluster.sync();
  // summed up by shares, and given to all
  for (int b = rank * (kBins / kCtas) + threadIdx.x; b < (rank + 1) * (kBins / kCtas); b += kThreads) {
    uint32_t n = 0;
    float place = 0.f;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      const Shared* o = cluster.map_shared_rank(&s, c);
      n += o->bins[b];
      place += static_cast<float>(o->places[b]);
    }
    place = n ? (place / n + 0.5f) * (1.f / 32.f) : 0.f;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      Shared* o = cluster.map_shared_rank(&s, c);
      o->all[b] = n;
      o->mean[b] = place;
    }
  }
  cluster.sync();
  make_plan(s, r, per_unit, P.vocab * 2.4e-10f);
  // Candidates of the borders' bins are collected, the others' weights summed up, for each segment between them.  (Behind the
  // third interval nothing counts: that there are three takes a filter that ends all.)
  const Plan& plan = s.plan;
  const float behind = plan.last == kBins - 1 ? INFINITY : (plan.last + 1) * 2048.f;
  // the least logit that can count, and less (of bf16 pieces the largest logit tells whether one does)
  const float least = fmaxf(top - behind / per_place * 1.00001f - fabsf(top) * 1e-6f, -3.4028235e38f);
  float from[3], upto[3];  // the intervals' places
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    from[j] = plan.begin[j] >= kBins ? INFINITY : plan.begin[j] * 2048.f;  // (there are fewer than three)
    upto[j] = plan.end[j] >= kBins - 1 ? INFINITY : (plan.end[j] + 1) * 2048.f;
  }
  int waiting = 0;
  uint32_t collected = 0;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    const float limit = fmaxf(plan.exact, round ? kExactAgain * per_unit : 0.f) * 2048.f;
    // of the segments, the places whose weights are summed up in fp32
    const float lo[3] = {limit, fmaxf(upto[0], limit), fmaxf(upto[1], limit)};
    const float hi[3] = {fminf(from[0], behind), fminf(from[1], behind), fminf(from[2], behind)};
    const bool third = lo[2] < hi[2];
    uint64_t mass[3] = {0, 0, 0}, light[3] = {0, 0, 0};
    const auto work_off = [&]() {
      while (__any_sync(0xffffffffu, waiting > 0)) {
        if (waiting > 0) {
          const float x = s.queue[--waiting][threadIdx.x], y = (top - x) * per_place;
          const uint64_t m = w.of(x, s.table);
          mass[0] += y < upto[0] ? m : 0;
          mass[1] += y >= upto[0] && y < upto[1] ? m : 0;
          mass[2] += y >= upto[1] ? m : 0;
        }
      }
    };
    each_raw<T>(P, row, first, step, [&](const Piece<T>& raw, int i0) {
      if (!__any_sync(0xffffffffu, piece_largest<T>(raw) >= least)) return;
      float x[kPiece];
      unpack_piece<T>(raw, x);
      float part[3] = {0.f, 0.f, 0.f};
      uint32_t apart = 0;  // not summed up here
#pragma unroll
      for (int e = 0; e < kPiece; e += 2) {
        const Two d = add2(two(x[e], x[e + 1]), two(-top));
        const float2 y2 = both(mul2(d, two(-per_place))), m2 = both(w.rounded(d));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float y = h ? y2.y : y2.x, m = h ? m2.y : m2.x;
          const bool p0 = y >= lo[0] && y < hi[0], p1 = y >= lo[1] && y < hi[1], p2 = third && y >= lo[2] && y < hi[2];
          if (p0) part[0] += m;
          if (p1) part[1] += m;
          if (p2) part[2] += m;
          if (!(p0 || p1 || p2)) apart |= 1u << (e + h);
        }
      }
      if (apart) {
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
          const float y = (top - x[e]) * per_place;
          if (!(apart >> e & 1) || !(y < behind) || !candidate(x[e])) continue;
          if ((y >= from[0] && y < upto[0]) || (y >= from[1] && y < upto[1]) || (y >= from[2] && y < upto[2])) {
            if (round == 0) {
              const uint32_t place = atomicAdd(&s.taken, 1u);
              if (place < kCollect) s.weights[place] = key_of(x[e], i0 + e);
            }
          } else {
            s.queue[waiting++][threadIdx.x] = x[e];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) light[k] += __float2ull_rn(part[k] * w.unit);
      if (__any_sync(0xffffffffu, waiting > kQueue - kPiece)) work_off();
    });
    work_off();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      // (5.25e-8 is 451 / 2^33)
      const uint64_t m = warp_sum(mass[k] + light[k] + (light[k] >> 20) * 451 / 8192);
      if ((threadIdx.x & 31) == 0 && m) atomicAdd(&head->segment[k], static_cast<unsigned long long>(m));
    }
    if (round == 0) {  // what this CTA has collected goes to the first one, in order of the bins
      __syncthreads();
      const uint32_t n = s.taken;
      if (threadIdx.x == 0 && n > 0) atomicAdd(&head->collected, n);
      for (uint32_t i = threadIdx.x; i < min(n, static_cast<uint32_t>(kCollect)); i += kThreads) {
        const uint64_t key = s.weights[i];
        const int bin = bin_of((top - logit_of(key)) * per_place);
        const uint32_t place = s.base[bin] + atomicAdd(&head->cursor[bin], 1u);
        if (place < kCollect) head->list[place] = key;
      }
    }
    cluster.sync();
    if (round == 0) {
      collected = head->collected;
      const int n = static_cast<int>(collected);
      // Ranking takes the square of a CTA's share of a bin, sorting less of many.  Equal logits, all in one bin, where ranking is slowest:
      // 64 rows of 128256, 4 CTAs each, 400, 800 and 1600 collected 43.6, 57.5 and 100 us ranked, 46.2, 52.7 and 72 sorted; 300 rows
      // of 32000, one each, 55, 94 and 247, and 50, 57 and 74
      const bool many = n > kCollect, few = !many && n * n <= kThreads * kThreads * kCtas;
      if (n <= 32) {
        if (rank == 0 && threadIdx.x < 32) rank_few(s, w, n);
      } else {
        if (few || (rank == 0 && !many)) {
          for (int i = threadIdx.x; i < n; i += kThreads) s.unsorted[i] = head->list[i];
          __syncthreads();
        }
        if (few) rank_share<kCtas>(s, head, w, per_place, n, rank);
        else if (rank == 0 && !many) sort_many(s, w, n);
        cluster.sync();  // (and the first CTA's memory has been read)
        if (many) break;
        if (rank == 0) {
          for (int i = threadIdx.x; i < n; i += kThreads) s.list[i] = s.sorted[i];
          __syncthreads();
        }
      }
    }
    if (rank == 0) {
      const int n = static_cast<int>(collected);
      const bool exact = round > 0;
      int left = 0;
      if (n > kFew) left = finish<false>(P, s, r, w, per_place, row, n, exact);
      else if (threadIdx.x < 32) left = finish<true>(P, s, r, w, per_place, row, n, exact);
      if (threadIdx.x == 0) s.unsure = left;
      if (left && threadIdx.x < 3) s.segment[threadIdx.x] = 0;
    }
    cluster.sync();
    const int left = head->unsure;
    cluster.sync();  // (the first CTA's memory has been read)
    if (left == 0) return;
    if (left == 2) break;
  }
  by_bisection<T, kCtas>(P, s, r, w, row, rank);
}

template <typename T, int kCtas>
int launch(const Params& p, int32_t rows, cudaStream_t s) {
  static uint64_t smem_set = 0;
  const int st = set_smem_once(reinterpret_cast<const void*>(sample_kernel<T, kCtas>), sizeof(Shared), &smem_set);
  return st ? st : cuda_status(launch_k(sample_kernel<T, kCtas>, dim3(rows * kCtas), dim3(kThreads), sizeof(Shared), s, p));
}

template <typename T>
int launch_rows(const Params& p, int32_t rows, int num_sms, cudaStream_t s) {
  // CTAs a row: as many as the SMs hold two of each, none with less than 1024 logits.  1, 2, 4 and 8 of them, all filters: one row of 32000 20.5,
  // 16.0, 13.6, 13.0 us, of 4000 13.0, 12.6, 12.4, 12.9; 64 of 128256 56, 36, 31, 47; 152 of 32000 27, 25, 51, 86; 304 of them 35, 49, 88, 160.
  // top-p alone: 33 rows of 50257 in fp32 44, 31, 24, 25; 64 of 128256 133, 77, 57, 65; 152 of 32000 37, 33, 56, 92; 304 of them 55, 63, 97, 174
  const int64_t room = 2 * static_cast<int64_t>(num_sms) / rows;
  const int most = static_cast<int>(room < 1 ? 1 : room > 8 ? 8 : room);
  if (most >= 8 && p.vocab >= 8192) return launch<T, 8>(p, rows, s);
  if (most >= 4 && p.vocab >= 4096) return launch<T, 4>(p, rows, s);
  if (most >= 2 && p.vocab >= 2048) return launch<T, 2>(p, rows, s);
  return launch<T, 1>(p, rows, s);
}

}  // namespace

int launch_sample(const SampleArgs& a, int num_sms, uint32_t* err, cudaStream_t s) {
  const Params p{a.logits, a.row_stride, a.temperature, a.top_p, a.min_p, a.uniform, a.top_k, a.tokens, a.logprobs, err, a.vocab,
                 weight_shift(a.vocab)};
  return a.dtype == PKV_F32 ? launch_rows<float>(p, a.num_seqs, num_sms, s) : launch_rows<__nv_bfloat16>(p, a.num_seqs, num_sms, s);
}

}  // namespace pkv
