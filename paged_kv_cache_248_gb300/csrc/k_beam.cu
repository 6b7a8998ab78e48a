// k_beam.cu -- beam search's step over the paged cache's requests: the best continuations
// of each request's beams out of their logits.
//
// Mathematics.  Beam w with token v scores cum_w + x_wv - log sum_u exp(x_wu).  Within a
// beam the order of the scores is the order of the logits, so one pass over a row can keep
// its running maximum and sum (the log-sum-exp) and its num_select best logits at once;
// only their few candidates meet the log-sum-exp, and each other, afterwards.
//
// scan_kernel.  A CTA reads a run of the rows in chunks of 64 bytes a thread, which stay in
// registers while the next chunk's are on their way: each value is loaded once, feeds its
// warp's sum of exponents (fp32, relative to the warp's maximum of the chunk), and is compared
// with a threshold.  The threshold comes from the threads' maxima of each chunk: if
// every one of the 8 warps has ceil(num_select / 8) threads whose maximum reaches t, then t is
// no better than the num_select-th best value, and nothing below it can be selected.  That
// costs a few warp reductions and lets a few dozen candidates through.  A candidate's 64-bit key
// is its value in an order-preserving form above the complement of its index, so that all keys
// differ and equal values rank by their index.  When the buffer is full all the same (equal or
// rising values) it is cut to its num_select best, the threshold becomes the last of them, and
// the rest of the chunk is looked at again.
//
// select_kernel.  One CTA per request joins the pieces: the log-sum-exp of each beam, joined in
// 64 bits, then the same collection over the pieces' candidates, ranked by 64-bit scores.
//
// Bound: reading the logits once (HBM); for one request, two launches and their latency.
#include "pkv_internal.cuh"
#include "ptx.cuh"
#include "softmax_row.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVals = 32;                         // values of a chunk per thread
constexpr int kChunk = kThreads * kVals;          // values of a chunk
constexpr int kMaxBeams = 64;
constexpr int kCap = 1536;                        // candidates collected between cuts
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving 32-bit form of a float (no NaN; -0 first becomes +0), larger is larger.
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered_bits(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t ordered_bits(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double from_ordered_bits(uint64_t o) {
  return __longlong_as_double(static_cast<long long>((o >> 63) ? o & ~(uint64_t(1) << 63) : ~o));
}

// Where the values of a chunk sit: whole 16-byte vectors when every row starts on a
// 16-byte boundary (kAligned), single values of consecutive threads otherwise.  One of the
// two for all rows of a call, and counted from the row's start, so that equal rows have
// equal sums wherever they lie and their ties stay ties.
struct ScanParams {
  const void* logits;
  const uint8_t* finished;
  uint64_t* keys;    // [rows][pieces][select], best first, 0: none
  float* ml;         // [rows][row_chunks][kWarps][2]: maximum, sum of exp(x - maximum) of a warp's values
  int64_t row_stride;
  int32_t vocab, select, pieces;
  int32_t row_chunks, run;  // chunks of a row; chunks of a CTA's run (the last run may be shorter)
  int64_t chunks;           // of all rows
};

constexpr uint32_t kOrderedNegInf = 0x007fffffu;  // ordered_bits(-inf)
constexpr float kLowest = -3.402823466e38f;      // what a candidate has at least

// A value that at least `need` threads of this warp reach (0: none), from their own.
__device__ __forceinline__ uint32_t reached_by(uint32_t mine, int need) {
  uint32_t top = 0;
#pragma unroll 1
  for (int i = 0; i < need; ++i) {
    top = __reduce_max_sync(0xffffffffu, mine);
    const uint32_t who = __ballot_sync(0xffffffffu, mine == top);
    if ((threadIdx.x & 31) == __ffs(who) - 1) mine = 0;
  }
  return top;
}

// A collected candidate: rank first by `hi`, then by `lo` (both larger is better).
struct Cand {
  uint64_t hi;
  uint32_t lo;
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ bool better(uint64_t a, uint64_t b) { return a > b; }

// Collected candidates in shared memory: 64-bit keys, or keys with a 32-bit tie-break.
struct Keys {
  uint64_t hi[kCap];
  __device__ __forceinline__ uint64_t get(int i) const { return hi[i]; }
  __device__ __forceinline__ void set(int i, uint64_t k) { hi[i] = k; }
};
struct Cands {
  uint64_t hi[kCap];
  uint32_t lo[kCap];
  __device__ __forceinline__ Cand get(int i) const { return Cand{hi[i], lo[i]}; }
  __device__ __forceinline__ void set(int i, const Cand& c) {
    hi[i] = c.hi;
    lo[i] = c.lo;
  }
};

// Cuts the n collected candidates to the k best, best first (all threads, with everything
// pushed); returns the new count.  Every candidate's rank is the number of better ones; few
// candidates are each ranked by several threads, which share the comparisons.
template <typename T, typename Buf>
__device__ int cut(Buf& buf, int* ranks, int n, int k) {
  if (n <= kThreads / 2) {
    int width = 32;
    while (width < n) width *= 2;
    const int i = threadIdx.x & (width - 1), step = kThreads / width;
    ranks[threadIdx.x] = 0;
    __syncthreads();
    T mine{};
    if (i < n) {
      mine = buf.get(i);
      int rank = 0;
#pragma unroll 4
      for (int j = threadIdx.x / width; j < n; j += step) rank += better(buf.get(j), mine) ? 1 : 0;
      if (rank > 0) atomicAdd(ranks + i, rank);
    }
    __syncthreads();
    if (threadIdx.x < n && ranks[threadIdx.x] < k) buf.set(ranks[threadIdx.x], mine);  // (i = threadIdx.x)
    __syncthreads();
    return min(n, k);
  }
  constexpr int kPer = kCap / kThreads;
  T mine[kPer];
  int rank[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x + j * kThreads;
    rank[j] = i < n ? 0 : kCap;
    if (i < n) mine[j] = buf.get(i);
  }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const T o = buf.get(i);
#pragma unroll
    for (int j = 0; j < kPer; ++j) rank[j] += better(o, mine[j]) ? 1 : 0;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (rank[j] < k) buf.set(rank[j], mine[j]);
  __syncthreads();
  return min(n, k);
}

// A chunk's values of one thread, as they were loaded.
template <typename T, bool kAligned>
struct Chunk;
template <bool kAligned>
struct Chunk<float, kAligned> {
  uint32_t w[kVals];
  __device__ __forceinline__ float value(int k) const { return __uint_as_float(w[k]); }
};
template <bool kAligned>
struct Chunk<__nv_bfloat16, kAligned> {
  uint32_t w[kVals / 2];
  __device__ __forceinline__ float value(int k) const {
    return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  }
};

// Index within the row of value k of the chunk that starts at `base`.
template <typename T, bool kAligned>
__device__ __forceinline__ int64_t index_of(int64_t base, int k) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  return kAligned ? base + (static_cast<int64_t>(k / kVec) * kThreads + threadIdx.x) * kVec + k % kVec
                  : base + static_cast<int64_t>(k) * kThreads + threadIdx.x;
}

template <typename T, bool kAligned>
__device__ __forceinline__ void load_chunk(Chunk<T, kAligned>& c, const T* x, int64_t base, int64_t end) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kWords = 4 / static_cast<int>(sizeof(T));  // values of a 32-bit word
  constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;  // -inf
  if (kAligned && base + kChunk <= end) {
#pragma unroll
    for (int v = 0; v < kVals / kVec; ++v) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + index_of<T, kAligned>(base, v * kVec)));
      c.w[4 * v] = w.x;
      c.w[4 * v + 1] = w.y;
      c.w[4 * v + 2] = w.z;
      c.w[4 * v + 3] = w.w;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < kVals; ++k) {
      const int64_t i = index_of<T, kAligned>(base, k);
      c.w[k] = i < end ? __ldg(reinterpret_cast<const uint32_t*>(x) + i) : kNone;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kVals; k += kWords) {
      const int64_t i = index_of<T, kAligned>(base, k), j = index_of<T, kAligned>(base, k + 1);
      const uint32_t lo = i < end ? __ldg(reinterpret_cast<const uint16_t*>(x) + i) : kNone & 0xffffu;
      const uint32_t hi = j < end ? __ldg(reinterpret_cast<const uint16_t*>(x) + j) : kNone & 0xffffu;
      c.w[k / kWords] = lo | hi << 16;
    }
  }
}

// The largest value, and that of each quarter (NaN does not count).
template <typename T, bool kAligned>
__device__ __forceinline__ float chunk_max(const Chunk<T, kAligned>& c, float (&tops)[4]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (sizeof(T) == 4) {
      float a = c.value(8 * g), b = c.value(8 * g + 1);
#pragma unroll
      for (int k = 2; k < 8; k += 2) {
        a = fmaxf(a, c.value(8 * g + k));
        b = fmaxf(b, c.value(8 * g + k + 1));
      }
      tops[g] = fmaxf(a, b);
    } else {
      auto pair = [&](int k) { return *reinterpret_cast<const __nv_bfloat162*>(&c.w[4 * g + k]); };
      const __nv_bfloat162 m = __hmax2(__hmax2(pair(0), pair(1)), __hmax2(pair(2), pair(3)));
      tops[g] = fmaxf(__low2float(m), __high2float(m));
    }
  }
  return fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads, 3) scan_kernel(const ScanParams P) {
  __shared__ Keys buf;
  __shared__ int s_count, s_rank[kThreads];
  __shared__ uint32_t s_reach[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int need = (P.select + kWarps - 1) / kWarps;
  const int64_t end = P.vocab;
  int64_t at_chunk = static_cast<int64_t>(blockIdx.x) * P.run;
  const int64_t last_chunk = min(at_chunk + P.run, P.chunks);
  // the run's part of one row after the other
#pragma unroll 1
  while (at_chunk < last_chunk) {
  const int64_t row = at_chunk / P.row_chunks;
  const int first = static_cast<int>(at_chunk - row * P.row_chunks);
  const int count = static_cast<int>(min(static_cast<int64_t>(P.row_chunks - first), last_chunk - at_chunk));
  at_chunk += count;
  // this part's number among the row's parts; the row's last part marks the numbers after it
  const int piece = static_cast<int>(blockIdx.x - row * P.row_chunks / P.run);
  const int pieces_here = first + count == P.row_chunks ? P.pieces - piece : 1;
  if (P.finished != nullptr && __ldg(P.finished + row) != 0) continue;
  const T* x = static_cast<const T*>(P.logits) + row * P.row_stride;
  int64_t base = static_cast<int64_t>(first) * kChunk;
  const int64_t stop = min(end, base + static_cast<int64_t>(count) * kChunk);
  if (threadIdx.x == 0) s_count = 0;
  __syncthreads();
  float2* ml = reinterpret_cast<float2*>(P.ml) + (row * P.row_chunks + first) * kWarps + warp;
  uint64_t floor_key = 0;  // keys up to this one are out
  bool exact = false;      // it is the num_select-th best key of a cut
  // (a 32-bit chunk takes as many registers as two 16-bit ones: it is not loaded ahead)
  constexpr bool kAhead = sizeof(T) == 2;
  Chunk<T, kAligned> cur, next;
  if (kAhead) load_chunk<T, kAligned>(next, x, base, end);
#pragma unroll 1
  for (; base < stop; base += kChunk) {
    if (kAhead) {
      cur = next;
      if (base + kChunk < stop) load_chunk<T, kAligned>(next, x, base + kChunk, end);
    } else {
      load_chunk<T, kAligned>(cur, x, base, end);
    }
    float tops[4];  // of the chunk's four vectors (quarters)
    const float top = chunk_max<T, kAligned>(cur, tops);
    if (floor_key == 0) {
      const uint32_t reach = reached_by(top > -INFINITY ? ordered_bits(top) : 0, need);
      if (lane == 0) s_reach[warp] = reach;
    }
    // The warp's maximum and sum, each chunk's and warp's for itself: rows are cut at different
    // places, and equal rows are to have equal sums all the same, so that their ties stay ties.
    // 2^(x c - r) with r = m c rounded; what the rounding left, m c - r, is put right in the sum,
    // and values near the maximum have exponents near 0, where they are exact.  (A NaN is no
    // maximum, but makes the sum NaN.)
    const uint32_t warp_top = __reduce_max_sync(0xffffffffu, top > -INFINITY ? ordered_bits(top) : 0);
    const float m = warp_top ? from_ordered_bits(warp_top) : -INFINITY;
    float a0 = 0.f, a1 = 0.f;
    if (fabsf(m) < 1e30f) {
      const float r = m * kLog2e;
#pragma unroll
      for (int k = 0; k < kVals; k += 2) {
        float ya, yb;
        ffma2(ya, yb, cur.value(k), cur.value(k + 1), kLog2e, -r);
        fadd2(a0, a1, ex2_approx(ya), ex2_approx(yb));
      }
      a0 *= exp2f(fmaf(-m, kLog2e, r));
      a1 *= exp2f(fmaf(-m, kLog2e, r));
    } else if (warp_top) {  // values that times log2(e) may not be finite (a type's lowest value)
#pragma unroll 1
      for (int k = 0; k < kVals; k += 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t i = index_of<T, kAligned>(base, k + e);
          if (i < end) a0 += ex2_approx((Elem<T>::to_f32(x[i]) - m) * kLog2e);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kVals; ++k) a0 += isnan(cur.value(k)) ? cur.value(k) : 0.f;
    }
    float l = a0 + a1;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) *ml = make_float2(m, l);
    ml += kWarps;
    if (floor_key == 0) {
      __syncthreads();
      // A value that 8 * need >= num_select threads reach: what is lower is out (keys with the
      // value itself stay in).  0 is no threshold: not every warp has enough values.
      uint32_t least = s_reach[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) least = min(least, s_reach[w]);
      if (least > 0) floor_key = (static_cast<uint64_t>(least) << 32) - 1;
      exact = false;
    }
    uint32_t todo = 0;
    if (top > -INFINITY && ordered_bits(top) >= static_cast<uint32_t>(floor_key >> 32)) {
      const float at_least =
          floor_key >> 32 > kOrderedNegInf ? from_ordered_bits(static_cast<uint32_t>(floor_key >> 32)) : kLowest;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (tops[g] >= at_least) {
#pragma unroll
          for (int k = 8 * g; k < 8 * g + 8; ++k) todo |= cur.value(k) >= at_least ? 1u << k : 0u;
        }
      }
    }
    while (true) {
      uint32_t again = 0;  // values that found no room
      while (todo != 0) {  // few: each is read once more, so that no register is indexed
        const int k = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t i = index_of<T, kAligned>(base, k);
        const uint64_t key = (static_cast<uint64_t>(ordered_bits(Elem<T>::to_f32(x[i]))) << 32) |
                             (0xffffffffu - static_cast<uint32_t>(i));
        if (key > floor_key) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kCap) buf.set(at, key);
          else again |= 1u << k;
        }
      }
      const int more = __syncthreads_or(again != 0);
      const int n = min(s_count, kCap);
      // The first chunk's exact threshold is worth a cut (later chunks pass few values then),
      // and so is a buffer that fills.
      if (more || n >= (exact ? 512 : P.select)) {
        __syncthreads();
        const int left = cut<uint64_t>(buf, s_rank, n, P.select);
        if (left == P.select) {
          floor_key = max(floor_key, buf.get(P.select - 1));
          exact = true;
        }
        if (threadIdx.x == 0) s_count = left;
        __syncthreads();
      }
      if (!more) break;
      todo = again;
    }
  }
  // the part's candidates, best first
  const int n = s_count;
  const int left = n > 0 ? cut<uint64_t>(buf, s_rank, n, P.select) : 0;
  uint64_t* out = P.keys + (row * P.pieces + piece) * P.select;
  for (int k = threadIdx.x; k < P.select * pieces_here; k += kThreads) out[k] = k < left ? buf.get(k) : 0;
  }
}

struct SelParams {
  const uint64_t* keys;
  const float* ml;
  const float* cum;
  const uint8_t* finished;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int32_t beams, vocab, select, pieces, sums, eos;  // sums: maxima and sums of a row
};

__global__ void __launch_bounds__(kThreads) select_kernel(const SelParams P) {
  __shared__ double s_lse[kMaxBeams], s_cum[kMaxBeams];
  __shared__ uint8_t s_done[kMaxBeams];
  __shared__ Cands buf;
  __shared__ __align__(16) uint32_t s_best[kThreads];
  __shared__ uint32_t s_floor;
  __shared__ int s_count, s_rank[kThreads];
  const int64_t n = blockIdx.x;
  const int W = P.beams, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_count = 0;
  grid_dep_wait();
  grid_dep_launch();
  // a warp per beam joins its sums
  for (int w = warp; w < W; w += kWarps) {
    const int64_t row = n * W + w;
    const bool done = P.finished != nullptr && __ldg(P.finished + row) != 0;
    const float2* ml = reinterpret_cast<const float2*>(P.ml) + row * P.sums;
    float m = -INFINITY;
    double sum = 0.0;
    if (!done) {
      for (int p = lane; p < P.sums; p += 32) m = fmaxf(m, __ldcg(ml + p).x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      for (int p = lane; p < P.sums; p += 32) {
        const float2 pml = __ldcg(ml + p);
        // (values of -inf alone add 0, or NaN where NaN was among them)
        sum += pml.x == -INFINITY ? pml.y : pml.y * exp2f((pml.x - m) * kLog2e);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (lane == 0) {
      s_cum[w] = __ldg(P.cum + row);
      s_done[w] = done ? 1 : 0;
      if (!done) s_lse[w] = m + log(sum);  // not finite: the beam has no candidates
    }
  }
  __syncthreads();
  const int lists = W * P.pieces;
  const int total = lists * P.select;
  // Candidate i: entry i / lists of list i % lists, so that consecutive threads hold the best
  // entries of all lists.  {0, 0}: none (ordered forms of finite scores are above 0).
  auto cand = [&](int i) -> Cand {
    Cand c{0, 0};
    const int entry = i / lists, list = i - entry * lists, w = list / P.pieces;
    if (s_done[w]) {
      if (entry == 0 && list == w * P.pieces && isfinite(s_cum[w]))
        c = Cand{ordered_bits(s_cum[w]), 0xffffffffu - (static_cast<uint32_t>(w) * P.vocab + P.eos)};
      return c;
    }
    const uint64_t key = __ldcg(P.keys + (n * lists + list) * P.select + entry);
    const double lse = s_lse[w];
    const double score = s_cum[w] + (static_cast<double>(from_ordered_bits(static_cast<uint32_t>(key >> 32))) - lse);
    if (key != 0 && isfinite(lse) && isfinite(score))
      c = Cand{ordered_bits(score), 0xffffffffu - (static_cast<uint32_t>(w) * P.vocab + (0xffffffffu - static_cast<uint32_t>(key)))};
    return c;
  };
  // A threshold on the upper half of the scores: the num_select-th largest of the threads'
  // maxima (the threads take the lists' best entries first, see cand).
  uint32_t best = 0;
  constexpr int kKeep = 4;  // candidates that a thread keeps in registers
  Cand kept[kKeep];
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kThreads;
    kept[j] = i < total ? cand(i) : Cand{0, 0};
    best = max(best, static_cast<uint32_t>(kept[j].hi >> 32));
  }
  Cand floor_c{0, 0xffffffffu};
  if (total > kThreads) {
    for (int i = threadIdx.x + kKeep * kThreads; i < total; i += kThreads)
      best = max(best, static_cast<uint32_t>(cand(i).hi >> 32));
    s_best[threadIdx.x] = best;
    if (threadIdx.x == 0) s_floor = 0;
    __syncthreads();
    int rank = 0;  // threads with a larger maximum, or the same and a lower index
#pragma unroll 4
    for (int t = 0; t < kThreads; t += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(s_best + t);
      rank += (o.x > best || (o.x == best && t < threadIdx.x)) + (o.y > best || (o.y == best && t + 1 < threadIdx.x)) +
              (o.z > best || (o.z == best && t + 2 < threadIdx.x)) + (o.w > best || (o.w == best && t + 3 < threadIdx.x));
    }
    if (rank == P.select - 1) s_floor = best;
    __syncthreads();
    if (s_floor > 0) floor_c.hi = (static_cast<uint64_t>(s_floor) << 32) - 1;
  } else if (P.select <= 32) {
    // few candidates: the num_select-th largest of any warp's will do, and the first warps,
    // which hold the lists' best entries, come close
    if (threadIdx.x == 0) s_floor = 0;
    __syncthreads();
    const uint32_t reach = reached_by(best, P.select);
    if (lane == 0 && reach > 0) atomicMax(&s_floor, reach);
    __syncthreads();
    if (s_floor > 0) floor_c.hi = (static_cast<uint64_t>(s_floor) << 32) - 1;
  }
  for (int base = 0; base < total; base += kKeep * kThreads) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
      const int i = base + threadIdx.x + j * kThreads;
      const Cand c = base == 0 ? kept[j] : (i < total ? cand(i) : Cand{0, 0});
      if (better(c, floor_c)) buf.set(atomicAdd(&s_count, 1), c);
    }
    __syncthreads();
    const int cnt = s_count;
    if (cnt + kKeep * kThreads > kCap && base + kKeep * kThreads < total) {
      __syncthreads();
      const int left = cut<Cand>(buf, s_rank, cnt, P.select);
      if (left == P.select) {
        const Cand last = buf.get(left - 1);
        if (better(last, floor_c)) floor_c = last;
      }
      if (threadIdx.x == 0) s_count = left;
    }
    __syncthreads();
  }
  const int cnt = s_count;
  const int left = cnt > 0 ? cut<Cand>(buf, s_rank, cnt, P.select) : 0;
  for (int k = threadIdx.x; k < P.select; k += kThreads) {
    const int64_t o = n * P.select + k;
    if (k < left) {
      const Cand c = buf.get(k);
      const uint32_t flat = 0xffffffffu - c.lo;
      P.out_scores[o] = static_cast<float>(from_ordered_bits(c.hi));
      P.out_parents[o] = static_cast<int32_t>(flat / static_cast<uint32_t>(P.vocab));
      P.out_tokens[o] = static_cast<int32_t>(flat % static_cast<uint32_t>(P.vocab));
    } else {
      P.out_scores[o] = -INFINITY;
      P.out_parents[o] = -1;
      P.out_tokens[o] = -1;
    }
  }
}

struct BeamPlan {
  int row_chunks, run, pieces, ctas;
  int64_t chunks;
  size_t key_bytes, bytes;
};

// All rows' chunks, one after the other, are cut into equal runs for as many CTAs as the GPU holds at
// once (kResident per SM); a row that lies in several runs has a part in each.
constexpr int kResident = 3;
BeamPlan beam_plan(int32_t num_seqs, int32_t beams, int32_t vocab, int32_t select, int num_sms) {
  BeamPlan b;
  const int64_t rows = static_cast<int64_t>(num_seqs) * beams;
  b.row_chunks = static_cast<int>((static_cast<int64_t>(vocab) + kChunk - 1) / kChunk);
  b.chunks = rows * b.row_chunks;
  const int64_t ctas = static_cast<int64_t>(kResident) * num_sms;
  b.run = static_cast<int>((b.chunks + ctas - 1) / ctas);
  b.ctas = static_cast<int>((b.chunks + b.run - 1) / b.run);
  b.pieces = (b.row_chunks + b.run - 2) / b.run + 1;  // runs that row_chunks chunks in a row can touch
  b.key_bytes = (static_cast<size_t>(rows) * b.pieces * select * sizeof(uint64_t) + 255) & ~static_cast<size_t>(255);
  b.bytes = b.key_bytes +
            ((static_cast<size_t>(b.chunks) * kWarps * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255));
  return b;
}

}  // namespace

size_t beam_workspace(int32_t num_seqs, int32_t beams, int32_t vocab, int32_t select, int num_sms) {
  return beam_plan(num_seqs, beams, vocab, select, num_sms).bytes;
}

int launch_beam_select(const BeamArgs& a, void* workspace, int num_sms, cudaStream_t s) {
  const BeamPlan b = beam_plan(a.num_seqs, a.beams, a.vocab, a.select, num_sms);
  ScanParams p{};
  p.logits = a.logits;
  p.finished = a.finished;
  p.keys = static_cast<uint64_t*>(workspace);
  p.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + b.key_bytes);
  p.row_stride = a.row_stride;
  p.vocab = a.vocab;
  p.select = a.select;
  p.pieces = b.pieces;
  p.row_chunks = b.row_chunks;
  p.run = b.run;
  p.chunks = b.chunks;
  const dim3 grid(static_cast<unsigned>(b.ctas));
  const int64_t elem = a.dtype == PKV_F32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && a.row_stride * elem % 16 == 0;
  cudaError_t e;
  if (a.dtype == PKV_F32)
    e = aligned ? launch_k(scan_kernel<float, true>, grid, dim3(kThreads), 0, s, p)
                : launch_k(scan_kernel<float, false>, grid, dim3(kThreads), 0, s, p);
  else
    e = aligned ? launch_k(scan_kernel<__nv_bfloat16, true>, grid, dim3(kThreads), 0, s, p)
                : launch_k(scan_kernel<__nv_bfloat16, false>, grid, dim3(kThreads), 0, s, p);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  SelParams q{p.keys, p.ml, a.cum, a.finished, a.out_scores, a.out_parents, a.out_tokens,
              a.beams, a.vocab, a.select, b.pieces, b.row_chunks * kWarps, a.eos};
  return cuda_status(launch_k(select_kernel, dim3(a.num_seqs), dim3(kThreads), 0, s, q));
}

}  // namespace pkv
