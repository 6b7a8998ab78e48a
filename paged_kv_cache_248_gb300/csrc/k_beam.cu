// k_beam.cu -- beam search's step over the paged cache's requests: the best continuations
// of each request's beams out of their logits.
//
// Mathematics.  Beam w with token v scores cum_w + x_wv - log sum_u exp(x_wu).  Rows are divided
// into blocks of 1024 consecutive logits, and one pass keeps of each block its maximum and the
// sum of its exponents.  The sums give the log-sum-exp of the rows; and the num_select best
// candidates lie in the num_select blocks whose maxima score best: of any other block, each
// candidate is beaten by those num_select maxima.  (Blocks whose maxima score alike are taken
// in order of their index, and so their candidates are, whose indices have the same order.)  So
// the second step reads num_select blocks a request again, and nothing else.
//
// scan_kernel.  A warp takes one block after the other: 32 values a lane in 16-byte loads, a
// maximum, the exponents relative to it and their sum in fp32.  No block shares anything with
// another, and equal rows have equal sums, so that their ties stay ties.  Bound: reading the
// logits (64 x 4 rows of 128256 bf16, 66 MB: 14.4 us, 67 % of a copy's rate; five CTAs an SM keep
// 80 KB of loads under way, and loading the next block ahead in registers as well was slower,
// because fewer warps fit).
//
// select_kernel.  One CTA per request joins the sums, ranks the blocks' maxima, collects what its
// best blocks hold, and ranks that, all by 64-bit scores.  Bound: the latency of its steps, 10
// to 12 thousand cycles for one request (of them 3100 for the sums, 3500 for the best blocks, 3600
// for reading these again, 1400 for the last ranking).  So little of it is done in 64 bits, of
// which an SM does two operations a cycle: joining the sums in doubles took 5400 cycles for 4 rows
// and 11400 for 16, which two fp32 values a sum, the second for what rounding lost, cut to 3100 and
// 3500.  A threshold that leaves few candidates comes from ranking 128 maxima against one another
// (600 cycles; a search bit by bit, with a barrier a bit, took 4000).
//
// Whole calls, on logits that are not in L2: 21.0 us for the batch above (HBM needs 9.7), 18.1 us for 9
// requests of 16 beams and 50257 fp32 logits, 32 selected, three in ten beams finished (3.1); on logits
// that are, as a model's last product leaves small ones, 17.6 and 15.4 us, and 7.7 us for one request of
// 4 beams and 32000 logits.
#include "pkv_internal.cuh"
#include "ptx.cuh"
#include "softmax_row.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVals = 32;                 // values of a block per lane
constexpr int kBlockVals = 32 * kVals;
constexpr int kSelThreads = 512;          // of the selection
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kGroups = kSelThreads / 4;   // groups of threads in a threshold
constexpr int kMaxBeams = 64;
constexpr int kCap = 1536;                // candidates collected between cuts
constexpr int kResident = 5;              // CTAs of the scan on an SM
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

// sum + lost += x, where lost gathers what the rounding of sum leaves out.
__device__ __forceinline__ void two_sum(float& sum, float& lost, float x) {
  const float s = __fadd_rn(sum, x), back = __fsub_rn(s, sum);
  lost += __fadd_rn(__fsub_rn(sum, __fsub_rn(s, back)), __fsub_rn(x, back));
  sum = s;
}
// The largest of the warp's values (NaN does not count).
__device__ __forceinline__ float max_over_warp(float x) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, x > -INFINITY ? ordered_bits(x) : 0);
  return top ? from_ordered_bits(top) : -INFINITY;
}

// A collected candidate: its score in the order-preserving form, then the complement of its
// index (both larger is better; no two candidates are equal).
struct Cand {
  uint64_t hi;
  uint32_t lo;
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
// Collected candidates in shared memory.
struct Cands {
  uint64_t hi[kCap];
  uint32_t lo[kCap];
  __device__ __forceinline__ Cand get(int i) const { return Cand{hi[i], lo[i]}; }
  __device__ __forceinline__ void set(int i, const Cand& c) {
    hi[i] = c.hi;
    lo[i] = c.lo;
  }
};

// What a selection needs in shared memory besides the candidates.
struct Scratch {
  uint32_t top[kGroups];
  int rank[kGroups];
  uint32_t least;
  int count;
};

// A threshold that `need` or more of the threads' values reach, and few more than `need` do (0:
// there are not as many): the need-th largest of the maxima of groups of four threads.
__device__ uint32_t reached_by(Scratch& s, int need, uint32_t value) {
  value = max(value, __shfl_xor_sync(0xffffffffu, value, 1));
  value = max(value, __shfl_xor_sync(0xffffffffu, value, 2));
  if ((threadIdx.x & 3) == 0) s.top[threadIdx.x >> 2] = value;
  if (threadIdx.x < kGroups) s.rank[threadIdx.x] = 0;
  if (threadIdx.x == 0) s.least = 0;
  __syncthreads();
  const int i = threadIdx.x % kGroups;
  const uint32_t mine = s.top[i];
  const uint4* other = reinterpret_cast<const uint4*>(s.top) + threadIdx.x / kGroups * (kGroups / 16);
  int reach = 0;  // of a quarter of the groups
#pragma unroll
  for (int j = 0; j < kGroups / 16; ++j) {
    const uint4 o = other[j];
    reach += (o.x >= mine) + (o.y >= mine) + (o.z >= mine) + (o.w >= mine);
  }
  atomicAdd(s.rank + i, reach);
  __syncthreads();
  if (threadIdx.x < kGroups && s.rank[i] >= need) atomicMax(&s.least, mine);
  __syncthreads();
  return s.least;
}

// Cuts the n collected candidates to the k best, best first (all threads, with everything
// pushed); returns the new count.  Every candidate's rank is the number of better ones; few
// candidates are each ranked by several threads, which share the comparisons, and of many the
// worse ones are left out by their upper halves first.
__device__ int cut(Cands& buf, Scratch& s, int n, int k) {
  constexpr int kPer = kCap / kSelThreads;
  for (int before = kCap + 1; n > kGroups && n < before;) {
    before = n;
    __syncthreads();  // (the count has been read)
    Cand mine[kPer];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x + j * kSelThreads;
      mine[j] = i < n ? buf.get(i) : Cand{0, 0};
      top = max(top, static_cast<uint32_t>(mine[j].hi >> 32));
    }
    if (threadIdx.x == 0) s.count = 0;
    const uint32_t least = reached_by(s, k, top);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (threadIdx.x + j * kSelThreads < n && static_cast<uint32_t>(mine[j].hi >> 32) >= least)
        buf.set(atomicAdd(&s.count, 1), mine[j]);
    __syncthreads();
    n = s.count;
    __syncthreads();
  }
  if (n <= kGroups) {
    int width = 32;
    while (width < n) width *= 2;
    const int i = threadIdx.x & (width - 1), step = kSelThreads / width;
    if (threadIdx.x < kGroups) s.rank[threadIdx.x] = 0;
    __syncthreads();
    Cand mine{0, 0};
    if (i < n) {
      mine = buf.get(i);
      int rank = 0;
#pragma unroll 4
      for (int j = threadIdx.x / width; j < n; j += step) rank += better(buf.get(j), mine) ? 1 : 0;
      if (rank > 0) atomicAdd(s.rank + i, rank);
    }
    __syncthreads();
    if (threadIdx.x < n && s.rank[i] < k) buf.set(s.rank[i], mine);  // (i = threadIdx.x)
    __syncthreads();
    return min(n, k);
  }
  Cand mine[kPer];  // (many with the same upper half)
  int rank[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x + j * kSelThreads;
    rank[j] = i < n ? 0 : kCap;
    mine[j] = i < n ? buf.get(i) : Cand{0, 0};
  }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const Cand o = buf.get(i);
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

struct ScanParams {
  const void* logits;
  const uint8_t* finished;
  float2* sums;      // [rows][row_blocks]: maximum, sum of exp(x - maximum)
  int64_t row_stride, blocks;  // blocks of all rows
  int32_t vocab, row_blocks;
};

// Index within its block of value k of this lane: whole 16-byte vectors when every row starts
// on a 16-byte boundary (kAligned), single values of consecutive lanes otherwise.
template <typename T, bool kAligned>
__device__ __forceinline__ int index_of(int k) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
  return kAligned ? (k / kVec * 32 + lane) * kVec + k % kVec : k * 32 + lane;
}

// A block's values of one lane, as they were loaded; what lies past the row's end is -inf.
template <typename T>
struct Values;
template <>
struct Values<float> {
  uint32_t w[kVals];
  __device__ __forceinline__ float get(int k) const { return __uint_as_float(w[k]); }
};
template <>
struct Values<__nv_bfloat16> {
  uint32_t w[kVals / 2];
  __device__ __forceinline__ float get(int k) const {
    return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  }
};

template <typename T, bool kAligned>
__device__ __forceinline__ void load_values(Values<T>& c, const T* x, int left) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  if (kAligned && left >= kBlockVals) {
#pragma unroll
    for (int v = 0; v < kVals / kVec; ++v) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + index_of<T, kAligned>(v * kVec)));
      c.w[4 * v] = w.x;
      c.w[4 * v + 1] = w.y;
      c.w[4 * v + 2] = w.z;
      c.w[4 * v + 3] = w.w;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < kVals; ++k) {
      const int i = index_of<T, kAligned>(k);
      c.w[k] = i < left ? __ldg(reinterpret_cast<const uint32_t*>(x) + i) : 0xff800000u;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kVals; k += 2) {
      const int i = index_of<T, kAligned>(k), j = index_of<T, kAligned>(k + 1);
      const uint32_t lo = i < left ? __ldg(reinterpret_cast<const uint16_t*>(x) + i) : 0xff80u;
      const uint32_t hi = j < left ? __ldg(reinterpret_cast<const uint16_t*>(x) + j) : 0xff80u;
      c.w[k / 2] = lo | hi << 16;
    }
  }
}

// The largest value (NaN does not count).
__device__ __forceinline__ float max_of(const Values<float>& c) {
  float a = c.get(0), b = c.get(1);
#pragma unroll
  for (int k = 2; k < kVals; k += 2) {
    a = fmaxf(a, c.get(k));
    b = fmaxf(b, c.get(k + 1));
  }
  return fmaxf(a, b);
}
__device__ __forceinline__ float max_of(const Values<__nv_bfloat16>& c) {
  auto pair = [&](int k) { return *reinterpret_cast<const __nv_bfloat162*>(&c.w[k]); };
  __nv_bfloat162 a = pair(0), b = pair(1);
#pragma unroll
  for (int k = 2; k < kVals / 2; k += 2) {
    a = __hmax2(a, pair(k));
    b = __hmax2(b, pair(k + 1));
  }
  a = __hmax2(a, b);
  return fmaxf(__low2float(a), __high2float(a));
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : kResident) scan_kernel(const ScanParams P) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
#pragma unroll 1
  for (int64_t n = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x; n < P.blocks; n += step) {
    const uint32_t row = static_cast<uint32_t>(n) / static_cast<uint32_t>(P.row_blocks);
    const int at = static_cast<int>(static_cast<uint32_t>(n) - row * P.row_blocks) * kBlockVals;
    if (P.finished != nullptr && __ldg(P.finished + row) != 0) continue;
    Values<T> c;
    const T* x = static_cast<const T*>(P.logits) + row * P.row_stride + at;
    load_values<T, kAligned>(c, x, P.vocab - at);
    const float top = max_of(c);
    const float m = max_over_warp(top);
    float a0 = 0.f, a1 = 0.f;
    if (fabsf(m) < 1e30f) {
      // 2^(x c - r) with r = m c rounded; what the rounding left, m c - r, is put right in the
      // sum, and values near the maximum have exponents near 0, where they are exact.  (A NaN
      // is no maximum, but makes the sum NaN.)
      const float r = m * kLog2e;
#pragma unroll
      for (int k = 0; k < kVals; k += 2) {
        float ya, yb;
        ffma2(ya, yb, c.get(k), c.get(k + 1), kLog2e, -r);
        fadd2(a0, a1, ex2_approx(ya), ex2_approx(yb));
      }
      a0 = (a0 + a1) * exp2f(fmaf(-m, kLog2e, r));
    } else if (m > -INFINITY) {  // values that times log2(e) may not be finite (a type's lowest value)
#pragma unroll 1
      for (int k = 0; k < kVals; ++k) {
        const int i = index_of<T, kAligned>(k);
        if (at + i < P.vocab) a0 += ex2_approx((Elem<T>::to_f32(x[i]) - m) * kLog2e);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kVals; ++k) a0 += isnan(c.get(k)) ? c.get(k) : 0.f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) a0 += __shfl_xor_sync(0xffffffffu, a0, d);
    if (lane == 0) P.sums[n] = make_float2(m, a0);
  }
}

struct SelParams {
  ScanParams scan;
  const float* cum;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int32_t beams, select, eos;
};

// Collects the num_select best of what `cand` gives for 0 .. total - 1 (all threads; {0, 0}:
// nothing) into buf, best first; returns how many there are.  What scores below the
// num_select-th largest of the threads' maxima is left out from the start.
template <typename F>
__device__ int best_of(Cands& buf, Scratch& s, int total, int select, F&& cand) {
  constexpr int kKeep = 2;  // candidates that a thread keeps in registers
  Cand kept[kKeep];
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = threadIdx.x + j * kSelThreads;
    kept[j] = i < total ? cand(i) : Cand{0, 0};
    best = max(best, static_cast<uint32_t>(kept[j].hi >> 32));
  }
  for (int i = threadIdx.x + kKeep * kSelThreads; i < total; i += kSelThreads)
    best = max(best, static_cast<uint32_t>(cand(i).hi >> 32));
  if (threadIdx.x == 0) s.count = 0;
  const uint32_t least = reached_by(s, select, best);
  Cand floor_c{least > 0 ? (static_cast<uint64_t>(least) << 32) - 1 : 0, 0xffffffffu};
#pragma unroll 1
  for (int base = 0; base < total; base += kKeep * kSelThreads) {
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
      const int i = base + threadIdx.x + j * kSelThreads;
      const Cand c = base == 0 ? kept[j] : (i < total ? cand(i) : Cand{0, 0});
      if (better(c, floor_c)) buf.set(atomicAdd(&s.count, 1), c);  // (room for all: kCap - 512 a turn)
    }
    __syncthreads();
    const int cnt = s.count;
    if (cnt + kKeep * kSelThreads > kCap && base + kKeep * kSelThreads < total) {
      __syncthreads();
      const int left = cut(buf, s, cnt, select);
      if (left == select && better(buf.get(left - 1), floor_c)) floor_c = buf.get(left - 1);
      if (threadIdx.x == 0) s.count = left;
    }
    __syncthreads();
  }
  const int cnt = s.count;
  return cnt > 0 ? cut(buf, s, cnt, select) : 0;
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelParams P) {
  __shared__ double s_off[kMaxBeams];  // what a row's values score besides themselves; not finite: it has no candidates
  __shared__ float s_top[kMaxBeams], s_log[kMaxBeams], s_least[kMaxBeams];
  __shared__ int s_exp[kMaxBeams];
  __shared__ uint8_t s_done[kMaxBeams];
  __shared__ Cands buf;
  __shared__ uint32_t s_blocks[64];
  __shared__ __align__(16) Scratch s;
  const int64_t n = blockIdx.x;
  const int W = P.beams, V = P.scan.vocab, per_row = P.scan.row_blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  const double cum = threadIdx.x < W ? __ldg(P.cum + n * W + threadIdx.x) : 0.f;
  // A warp per beam joins its sums, each with what its rounding lost beside it.
  for (int w = warp; w < W; w += kSelWarps) {
    const int64_t row = n * W + w;
    const bool done = P.scan.finished != nullptr && __ldg(P.scan.finished + row) != 0;
    const float2* sums = P.scan.sums + row * per_row;
    float m = -INFINITY, sum = 0.f, lost = 0.f;
    if (!done) {
      for (int p = lane; p < per_row; p += 32) m = fmaxf(m, sums[p].x);
      m = max_over_warp(m);
      for (int p = lane; p < per_row; p += 32) {
        const float2 part = sums[p];
        // (values of -inf alone add 0, or NaN where NaN was among them)
        two_sum(sum, lost, part.x == -INFINITY ? part.y : part.y * exp2f((part.x - m) * kLog2e));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        lost += __shfl_xor_sync(0xffffffffu, lost, d);
        two_sum(sum, lost, __shfl_xor_sync(0xffffffffu, sum, d));
      }
    }
    if (lane == 0) {
      // log(sum) = e ln 2 + log1p(f - 1) with f in [0.75, 1.5): the second part, below 0.41, is
      // off by 2^-25 of 1 or so in fp32, and the first is left to 64 bits
      const int e = (static_cast<int>(__float_as_uint(sum)) - 0x3f400000) >> 23;
      const bool usual = sum > 0.f && sum < INFINITY;
      const float down = __int_as_float((127 - e) << 23);
      s_done[w] = done ? 1 : 0;
      s_top[w] = m;
      s_exp[w] = e;
      s_log[w] = usual ? log1pf(fmaf(sum, down, -1.f) + lost * down) : NAN;
    }
  }
  __syncthreads();
  if (threadIdx.x < W) {
    const int w = threadIdx.x;
    s_off[w] = s_done[w] ? cum : cum - (s_top[w] + (s_exp[w] * 0.6931471805599453 + s_log[w]));
  }
  __syncthreads();
  // A value's score in its order-preserving form, 0 where it is no candidate (those of finite
  // scores are above 0).
  auto score_of = [&](int w, float x) -> uint64_t {
    const double score = s_off[w] + static_cast<double>(x);
    return isfinite(score) ? ordered_bits(score) : 0;
  };
  // the best blocks: a finished beam is one of one candidate, its first
  const int blocks = best_of(buf, s, W * per_row, P.select, [&](int i) -> Cand {
    const int w = i / per_row;
    uint64_t hi;
    if (s_done[w]) hi = i == w * per_row ? score_of(w, 0.f) : 0;
    else hi = score_of(w, P.scan.sums[n * W * per_row + i].x);
    return hi ? Cand{hi, ~static_cast<uint32_t>(i)} : Cand{0, 0};
  });
  // what they hold, as far as it scores as the last of their maxima
  Cand floor_c{0, 0xffffffffu};
  if (blocks == P.select) floor_c.hi = buf.get(blocks - 1).hi - 1;
  if (threadIdx.x < blocks) s_blocks[threadIdx.x] = ~buf.get(threadIdx.x).lo;
  // a little below beam w's value that has the floor's score
  auto least_value = [&](int w) -> float {
    if (!floor_c.hi) return -3.402823466e38f;
    const double at = from_ordered_bits(floor_c.hi), t = at - s_off[w];
    return fmaxf(-3.402823466e38f, static_cast<float>(t - (1e-5 * fabs(t) + 1e-15 * (fabs(at) + fabs(s_off[w])) + 1e-30)));
  };
  if (threadIdx.x < W) s_least[threadIdx.x] = least_value(threadIdx.x);
  __syncthreads();
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
#pragma unroll 1
  for (int b0 = 0; b0 < blocks; b0 += kSelWarps) {
    uint32_t todo = 0;
    int w = 0, at = 0;
    const T* x = nullptr;
    const bool have = b0 + warp < blocks;
    Values<T> c;
    if (have) {
      const int i = static_cast<int>(s_blocks[b0 + warp]);
      w = i / per_row;
      at = (i - w * per_row) * kBlockVals;
      x = static_cast<const T*>(P.scan.logits) + (n * W + w) * P.scan.row_stride + at;
      if (!s_done[w]) load_values<T, kAligned>(c, x, V - at);
    }
    if (b0 == 0 && !floor_c.hi) {  // fewer blocks than asked for: the lanes' best values give a floor
      uint64_t top = 0;
      if (have && s_done[w]) top = lane == 0 ? score_of(w, 0.f) : 0;
      else if (have) top = score_of(w, max_of(c));
      const uint32_t least = reached_by(s, P.select, static_cast<uint32_t>(top >> 32));
      if (least > 0) {
        floor_c.hi = (static_cast<uint64_t>(least) << 32) - 1;
        if (threadIdx.x < W) s_least[threadIdx.x] = least_value(threadIdx.x);
        __syncthreads();
      }
    }
    if (have) {
      if (s_done[w]) {
        todo = lane == 0 ? 1 : 0;
      } else {
        const float least = s_least[w];
#pragma unroll
        for (int k = 0; k < kVals; ++k) todo |= c.get(k) >= least ? 1u << k : 0u;
      }
    }
    while (true) {
      uint32_t again = 0;  // values that found no room
      while (todo != 0) {  // few: each is read once more, so that no register is indexed
        const int k = __ffs(todo) - 1;
        todo &= todo - 1;
        const int i = index_of<T, kAligned>(k);
        const Cand c = s_done[w] ? Cand{score_of(w, 0.f), ~(static_cast<uint32_t>(w) * V + P.eos)}
                                 : Cand{score_of(w, Elem<T>::to_f32(x[i])), ~(static_cast<uint32_t>(w) * V + at + i)};
        if (c.hi && better(c, floor_c)) {
          const int to = atomicAdd(&s.count, 1);
          if (to < kCap) buf.set(to, c);
          else again |= 1u << k;
        }
      }
      const int more = __syncthreads_or(again != 0);
      const int cnt = min(s.count, kCap);
      __syncthreads();
      if (more) {
        const int left = cut(buf, s, cnt, P.select);
        if (left == P.select && better(buf.get(left - 1), floor_c)) floor_c = buf.get(left - 1);
        if (threadIdx.x == 0) s.count = left;
        __syncthreads();
      }
      if (!more) break;
      todo = again;
    }
  }
  const int cnt = s.count;
  const int left = cnt > 0 ? cut(buf, s, cnt, P.select) : 0;
  for (int k = threadIdx.x; k < P.select; k += kSelThreads) {
    const int64_t o = n * P.select + k;
    if (k < left) {
      const Cand c = buf.get(k);
      const uint32_t flat = ~c.lo;
      P.out_scores[o] = static_cast<float>(from_ordered_bits(c.hi));
      P.out_parents[o] = static_cast<int32_t>(flat / static_cast<uint32_t>(V));
      P.out_tokens[o] = static_cast<int32_t>(flat % static_cast<uint32_t>(V));
    } else {
      P.out_scores[o] = -INFINITY;
      P.out_parents[o] = -1;
      P.out_tokens[o] = -1;
    }
  }
}

template <typename T, bool kAligned>
int launch_typed(const SelParams& q, int32_t num_seqs, int num_sms, cudaStream_t s) {
  const int64_t want = (q.scan.blocks + kWarps - 1) / kWarps, most = static_cast<int64_t>(num_sms) * kResident;
  const int st = cuda_status(launch_k(scan_kernel<T, kAligned>, dim3(static_cast<unsigned>(want < most ? want : most)),
                                      dim3(kThreads), 0, s, q.scan));
  if (st) return st;
  return cuda_status(launch_k(select_kernel<T, kAligned>, dim3(num_seqs), dim3(kSelThreads), 0, s, q));
}

int64_t row_blocks(int32_t vocab) { return (static_cast<int64_t>(vocab) + kBlockVals - 1) / kBlockVals; }

}  // namespace

size_t beam_workspace(int32_t num_seqs, int32_t beams, int32_t vocab, int32_t, int) {
  return (static_cast<size_t>(num_seqs) * beams * row_blocks(vocab) * sizeof(float2) + 255) & ~static_cast<size_t>(255);
}

int launch_beam_select(const BeamArgs& a, void* workspace, int num_sms, cudaStream_t s) {
  SelParams q{};
  q.scan.logits = a.logits;
  q.scan.finished = a.finished;
  q.scan.sums = static_cast<float2*>(workspace);
  q.scan.row_stride = a.row_stride;
  q.scan.vocab = a.vocab;
  q.scan.row_blocks = static_cast<int32_t>(row_blocks(a.vocab));
  q.scan.blocks = static_cast<int64_t>(a.num_seqs) * a.beams * q.scan.row_blocks;
  q.cum = a.cum;
  q.out_scores = a.out_scores;
  q.out_parents = a.out_parents;
  q.out_tokens = a.out_tokens;
  q.beams = a.beams;
  q.select = a.select;
  q.eos = a.eos;
  const int64_t elem = a.dtype == PKV_F32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && a.row_stride * elem % 16 == 0;
  if (a.dtype == PKV_F32)
    return aligned ? launch_typed<float, true>(q, a.num_seqs, num_sms, s)
                   : launch_typed<float, false>(q, a.num_seqs, num_sms, s);
  return aligned ? launch_typed<__nv_bfloat16, true>(q, a.num_seqs, num_sms, s)
                 : launch_typed<__nv_bfloat16, false>(q, a.num_seqs, num_sms, s);
}

}  // namespace pkv
