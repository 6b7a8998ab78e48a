// tree_merge.cuh -- joining the parts of a unit that several runs of the tree attention worked on.
//
// Part p of a unit leaves, for each of its rows, an accumulator o_p, a maximum m_p (in log2 units)
// and a sum l_p over its keys; with M = max m_p the row is sum 2^(m_p - M) o_p / sum 2^(m_p - M) l_p,
// added up in the order of the keys.  The rows of a unit are shared out among the CTAs of its
// parts.  Up to 16 parts a warp joins a row's; of more, the CTA's warps join an eighth each, and one
// of them the eighths, in order.  Loads of four parts are under way at once, since latency is what
// this costs (2 requests of 8000 and 15000 keys, 8 nodes, 8 / 2 heads, up to 100 parts: 18.5 us a call,
// and 20.8 with a warp for all of a row's parts).
#pragma once
#include "pkv_internal.cuh"

namespace pkv {

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kManyParts = 16;
// CTAs per part.  (A unit has two parts or more, so that this makes for one turn of its rows, or two; twice
// as many CTAs take longer to start than they save: 102.1 instead of 101.5 us for 64 requests of 16 nodes.)
inline unsigned merge_ctas(int rows_cap) { return static_cast<unsigned>(rows_cap > 128 ? 4 : (rows_cap + 31) / 32); }

// What a part of a unit that is cut leaves besides its rows, at the slot of its partials.
struct alignas(16) Cut {
  int32_t parts;  // of the unit; 0: nothing is cut here
  int32_t share;  // which one this is
  int32_t t0, head;
  int32_t first[2], rows[2];  // of up to two row tiles
};

// Row r of part p of the unit that begins in run `begin`: a run's second slot holds the unit that it
// begins, its first the one that it goes on with.
__device__ __forceinline__ int64_t part_row(int begin, int p, int rows_cap, int r) {
  return static_cast<int64_t>(2 * (begin + p) + (p == 0 ? 1 : 0)) * rows_cap + r;
}

// A lane's E columns of a row, joined from some of its parts.
template <int E>
struct Joined {
  float m = -INFINITY, l = 0.f, o[E] = {};
  bool bad = false;  // a part with a bad block id (marked by a sum of -1)

  // Adds parts whose maxima are at most `top`; what has been added so far is rescaled to it.
  __device__ __forceinline__ void raise(float top) {
    const float f = m == top ? 1.f : exp2f(m - top);
    m = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
  }
  __device__ __forceinline__ void add(float pm, float pl, const float (&po)[E]) {
    // (a part without a maximum saw nothing, or nothing but NaN, which its sum says)
    const float w = pm == -INFINITY ? pl * 0.f : exp2f(pm - m);
    if (w != 0.f) {
      l = fmaf(pl, w, l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(po[e], w, o[e]);
    }
  }
};

// Parts p0 .. p1 - 1 of a row (a warp).
template <int E>
__device__ __forceinline__ Joined<E> join_parts(const float* part_o, const float* part_ml, int begin, int rows_cap, int row,
                                                int p0, int p1) {
  constexpr int kAtOnce = 4;
  const int lane = threadIdx.x & 31;
  Joined<E> j;
#pragma unroll 1
  for (int p = p0; p < p1; p += kAtOnce) {
    float2 ml[kAtOnce];
    float o[kAtOnce][E];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) o[k][e] = 0.f;
      if (p + k < p1) {
        const int64_t at = part_row(begin, p + k, rows_cap, row);
        ml[k] = __ldcg(reinterpret_cast<const float2*>(part_ml) + at);
        const float* src = part_o + (at * 32 + lane) * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          if (E % 4 == 0) {
            if (e % 4 == 0) {
              const float4 y = __ldcg(reinterpret_cast<const float4*>(src + e));
              o[k][e] = y.x;
              o[k][e + 1] = y.y;
              o[k][(e + 2) % E] = y.z;
              o[k][(e + 3) % E] = y.w;
            }
          } else {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(src + e));
            o[k][e] = y.x;
            o[k][e + 1] = y.y;
          }
        }
      }
    }
    float top = j.m;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, ml[k].x);
    j.raise(top);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      j.bad |= ml[k].y == -1.f;
      j.add(ml[k].x, ml[k].y, o[k]);
    }
  }
  return j;
}

// Joins this CTA's rows of the unit whose part the record at slot blockIdx.x is (all threads); calls
// store(cut, row, joined) by whole warps, where live(cut, row) says that the row is one.
template <int E, typename Live, typename Store>
__device__ __forceinline__ void join_rows(const Cut* cuts, const float* part_o, const float* part_ml, int rows_cap, Live&& live,
                                          Store&& store) {
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps], s_o[kMergeWarps][32 * E];
  __shared__ int s_bad[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4* rec = reinterpret_cast<const int4*>(cuts + blockIdx.x);
  const int4 c0 = __ldcg(rec), c1 = __ldcg(rec + 1);
  const Cut cut{c0.x, c0.y, c0.z, c0.w, {c1.x, c1.y}, {c1.z, c1.w}};
  const int begin = static_cast<int>(blockIdx.x >> 1) - cut.share;
  if (cut.parts < 2 || begin < 0 || begin + cut.parts > static_cast<int>(gridDim.x >> 1)) return;
  const bool split = cut.parts > kManyParts;
  const int rows_at_once = split ? 1 : kMergeWarps, place = split ? 0 : warp;
  const int p0 = split ? cut.parts * warp / kMergeWarps : 0;
  const int p1 = split ? cut.parts * (warp + 1) / kMergeWarps : cut.parts;
  const int step = cut.parts * gridDim.y * rows_at_once;
#pragma unroll 1
  for (int row = (cut.share * gridDim.y + blockIdx.y) * rows_at_once + place; row < rows_cap; row += step) {
    if (!live(cut, row)) continue;
    Joined<E> j = join_parts<E>(part_o, part_ml, begin, rows_cap, row, p0, p1);
    if (split) {
      if (lane == 0) {
        s_m[warp] = j.m;
        s_l[warp] = j.l;
        s_bad[warp] = j.bad;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = j.o[e];
      __syncthreads();
      if (warp == 0) {
        float top = -INFINITY;
#pragma unroll 1
        for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, s_m[w]);
        j.raise(top);  // (the first eighth is the warp's own)
#pragma unroll 1
        for (int w = 1; w < kMergeWarps; ++w) {
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = s_o[w][lane * E + e];
          j.add(s_m[w], s_l[w], o);
          j.bad |= s_bad[w] != 0;
        }
      }
    }
    if (place == warp || warp == 0) store(cut, row, j);
    if (split) __syncthreads();
  }
}

}  // namespace pkv
