// k_sample.cu -- tokens drawn from logits, with temperature, top-k, min-p and top-p.
//
// Mathematics.  The candidates of a row in order (larger logit first, of equal ones the lower index) have the
// weights w = exp((x - max) / T).  Every filter keeps a beginning of that order: the first k; those with
// w >= min_p; the shortest with mass >= top_p of what is left.  The token is the first whose cumulative
// weight exceeds u times the kept mass.  Whether a sum of a hundred thousand weights lies above or below
// a border is decided by its last digits, so weights are whole numbers: w 2^S rounded, right to about 2^-40
// of w (weight.cuh), and sums of them exact, in any order.
//
// Work.  A row belongs to a cluster of CTAs, which go through it three times (twice from L2):
//   1. its largest logit;
//   2. how many candidates fall into each of 4096 bins of (max - x) / T, 1/128 of a power of two wide.  That bounds
//      every mass to 0.6 %, and so tells for each border (the end of top-k and min-p, of top-p, the token) a few
//      bins in which it must lie;
//   3. the candidates of those bins are collected in the cluster's first CTA, and the others' exact weights summed
//      up between them.
// The first CTA sorts what was collected (hundreds, as a rule) and finds the borders exactly.  With top-k or min-p
// nothing behind their end is looked at closely, so that no weight but the collected ones' is ever computed.
// Where more than 8192 candidates lie in the borders' bins (rows of equal logits), borders are found by bisection
// of the keys instead, a pass over the row each.
//
// Bound: latency.  Three passes and five cluster barriers for one row; for many rows the exact weights of rows
// without top-k or min-p (about 40 instructions a logit).
#include <cooperative_groups.h>

#include "pkv_internal.cuh"
#include "weight.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 4096, kPerThread = kBins / kThreads;
constexpr float kBinsPerUnit = 128.f;
constexpr int kCollect = 8192;
constexpr int kGather = 255, kIgnore = 254;  // of a bin: its candidates are collected; lie behind everything

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

// What the first CTA finds out about the bins: up to three disjoint intervals of bins that are collected.
struct Plan {
  int32_t count;         // intervals
  int32_t begin[3], end[3];  // bins [begin, end]
  int32_t last;          // bins behind it are ignored
  int32_t rank[3];       // candidate number e of the list, in interval j, is number rank[j] + e of the row
};

struct Shared {
  union {
    struct {
      uint32_t bins[kBins];   // of this CTA
      uint32_t total[kBins];  // of the row (first CTA)
    };
    uint64_t list[kCollect];  // keys (first CTA)
  };
  uint8_t kind[kBins];  // of a bin: kGather, kIgnore, or how many intervals come before it
  uint64_t table[256];
  unsigned long long best[16], finite[16];  // of each CTA: its least key; its candidates
  unsigned long long segment[4];            // masses of what is not collected, between the intervals (first CTA)
  unsigned long long warp_u64[kWarps + 1];
  float warp_lo[kWarps], warp_hi[kWarps];
  uint32_t warp_n[kWarps];
  int32_t found[8];
  float bound[4];
  uint32_t collected;  // (first CTA)
  Plan plan;           // (first CTA)
  unsigned long long sum[2], least, most;  // of a pass of the bisection
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

// Calls f(x, i) for this thread's logits of the row (those of 16-byte pieces `first`, first + step, ...), of which
// several pieces are on their way at once.
template <typename T, typename F>
__device__ __forceinline__ void each(const Params& P, int64_t row, int first, int step, F&& f) {
  constexpr int kVec = 16 / sizeof(T), kAtOnce = 4;
  const T* p = static_cast<const T*>(P.logits) + row * P.stride;
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));  // piece 0 begins so much before
  const int pieces = (skew + P.vocab + kVec - 1) / kVec;
  const uint4* base = reinterpret_cast<const uint4*>(p - skew);
#pragma unroll 1
  for (int v0 = first; v0 < pieces; v0 += kAtOnce * step) {
    uint4 raw[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int v = v0 + k * step, i0 = v * kVec - skew;
      raw[k] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);  // NaN: no candidates
      if (v >= pieces) continue;
      if (i0 >= 0 && i0 + kVec <= P.vocab) {
        raw[k] = __ldg(base + v);
      } else {  // a piece that the row has a part of
        uint32_t* w = reinterpret_cast<uint32_t*>(&raw[k]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          if (i0 + e < 0 || i0 + e >= P.vocab) continue;
          if constexpr (sizeof(T) == 4) {
            w[e] = __float_as_uint(Elem<T>::to_f32(p[i0 + e]));
          } else {
            const uint32_t h = __float_as_uint(Elem<T>::to_f32(p[i0 + e])) >> 16;
            w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | h << 16 : (w[e / 2] & 0xffff0000u) | h;
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i0 = (v0 + k * step) * kVec - skew;
      const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float x = __uint_as_float(sizeof(T) == 4 ? w[e % 4] : e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        f(x, i0 + e);
      }
    }
  }
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

// The borders' bins, from the counts (the first CTA; candidates: all of the row).
__device__ __forceinline__ void make_plan(Shared& s, const Row& r, uint32_t candidates) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = threadIdx.x * kPerThread;
  // this thread's bins: candidates up to each, and bounds of their mass
  uint32_t n[kPerThread];
  float lo[kPerThread], hi[kPerThread];
  uint32_t cn = 0;
  float cl = 0.f, ch = 0.f;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = b0 + k;
    const uint32_t here = s.total[b];
    // (a bin number is off by up to 2^-10, and the sums of bounds by 2^-13)
    const float top = exp2f(static_cast<float>(-b) * (1.f / kBinsPerUnit));
    cn += here;
    ch += here * (top * (1.f + 1.f / 4096.f));
    cl += b == kBins - 1 ? 0.f : here * (top * (0.99459944f * (1.f - 1.f / 4096.f)));  // 2^(-1/128)
    n[k] = cn;
    lo[k] = cl;
    hi[k] = ch;
  }
  uint32_t in = cn;
  float il = cl, ih = ch;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, in, d);
    const float yl = __shfl_up_sync(0xffffffffu, il, d), yh = __shfl_up_sync(0xffffffffu, ih, d);
    if (lane >= d) {
      in += y;
      il += yl;
      ih += yh;
    }
  }
  if (lane == 31) {
    s.warp_n[warp] = in;
    s.warp_lo[warp] = il;
    s.warp_hi[warp] = ih;
  }
  if (threadIdx.x < 8) s.found[threadIdx.x] = kBins - 1;
  __syncthreads();
  uint32_t bn = in - cn;
  float bl = il - cl, bh = ih - ch, all_lo = 0.f, all_hi = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      bn += s.warp_n[w];
      bl += s.warp_lo[w];
      bh += s.warp_hi[w];
    }
    all_lo += s.warp_lo[w];
    all_hi += s.warp_hi[w];
  }
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    n[k] += bn;
    // (the differences above may round to below what was; the margins cover it)
    lo[k] += bl;
    hi[k] += bh;
  }
  // The first bin up to which more than `x` lies, by counts (0), by the lower (1) or the upper bounds (2): found[at].
  const auto search = [&](int at, int what, float x, uint32_t count) {
#pragma unroll
    for (int k = kPerThread - 1; k >= 0; --k)
      if (what == 0 ? n[k] >= count : (what == 1 ? lo[k] : hi[k]) > x) atomicMin(&s.found[at], b0 + k);
  };
  const bool cut_k = r.top_k > 0 && static_cast<uint32_t>(r.top_k) < candidates, cut_m = r.min_p > 0.f;
  if (cut_k) search(0, 0, 0.f, static_cast<uint32_t>(r.top_k));
  __syncthreads();
  int a1 = kBins, e1 = kBins - 1;  // the end of top-k and min-p
  if (cut_k) a1 = e1 = s.found[0];
  if (cut_m) {
    const int at = static_cast<int>(fminf(-log2f(r.min_p) * kBinsPerUnit, kBins - 1.f));
    a1 = min(a1, max(at - 1, 0));
    e1 = min(e1, min(at + 1, kBins - 1));
  }
  const bool cut1 = cut_k || cut_m;
  // the mass up to there: bounds
  if (cut1) {
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      if (b0 + k == a1 - 1) s.bound[0] = lo[k];
      if (b0 + k == e1) s.bound[1] = hi[k];
    }
    if (threadIdx.x == 0 && a1 == 0) s.bound[0] = 0.f;
    __syncthreads();
  }
  float z_lo = cut1 ? s.bound[0] : all_lo, z_hi = cut1 ? s.bound[1] : all_hi;
  z_lo *= 0.9999f;
  z_hi *= 1.0001f;
  // the end of top-p
  int a2 = kBins, e2 = e1;
  const bool cut_p = r.top_p < 1.f;
  if (cut_p) {
    search(1, 2, r.top_p * z_lo * 0.9999f, 0);
    search(2, 1, r.top_p * z_hi * 1.0001f, 0);
    __syncthreads();
    a2 = min(s.found[1], e1);
    e2 = min(s.found[2], e1);
    z_lo *= r.top_p;
    z_hi = fminf(z_hi, r.top_p * z_hi + 1.001f * exp2f(static_cast<float>(-a2) * (1.f / kBinsPerUnit)));
  }
  search(3, 2, r.u * z_lo * 0.9999f, 0);
  search(4, 1, r.u * z_hi * 1.0001f, 0);
  __syncthreads();
  if (threadIdx.x == 0) {
    int begin[3] = {}, end[3] = {}, m = 0;
    const auto add = [&](int a, int e) {  // (in order of their beginnings)
      if (m > 0 && a <= end[m - 1] + 1) {
        end[m - 1] = max(end[m - 1], e);
        return;
      }
      begin[m] = a;
      end[m++] = e;
    };
    const int a3 = min(s.found[3], e2), e3 = min(s.found[4], e2);
    // the token comes before the end of top-p, and that before the end of the others; their windows may overlap
    int a[3] = {a3, a2, a1}, e[3] = {e3, e2, e1};
    bool on[3] = {true, cut_p, cut1};
    for (int i = 0; i < 3; ++i)
      for (int k = i + 1; k < 3; ++k)
        if (on[k] && (!on[i] || a[k] < a[i])) {
          const int x = a[i], y = e[i];
          const bool z = on[i];
          a[i] = a[k], e[i] = e[k], on[i] = on[k];
          a[k] = x, e[k] = y, on[k] = z;
        }
    for (int i = 0; i < 3; ++i)
      if (on[i]) add(a[i], max(a[i], e[i]));
    s.plan.count = m;
    for (int i = 0; i < 3; ++i) {
      s.plan.begin[i] = i < m ? begin[i] : kBins;
      s.plan.end[i] = i < m ? end[i] : kBins;
    }
    s.plan.last = cut1 ? e1 : kBins - 1;
  }
  __syncthreads();
  // candidates before an interval that are not collected
#pragma unroll
  for (int k = 0; k < kPerThread; ++k)
    for (int j = 0; j < 3; ++j) {
      if (s.plan.begin[j] == b0 + k) s.plan.rank[j] = static_cast<int32_t>(n[k] - s.total[b0 + k]);
      if (s.plan.end[j] == b0 + k) s.found[5 + j] = static_cast<int32_t>(n[k]);
    }
  __syncthreads();
  if (threadIdx.x == 0) {
    int collected = 0;
    for (int j = 0; j < s.plan.count; ++j) {
      const int before = s.plan.rank[j];
      s.plan.rank[j] -= collected;
      collected += s.found[5 + j] - before;
    }
    s.collected = 0;
    for (int k = 0; k < 4; ++k) s.segment[k] = 0;
  }
}

// Sorts list[0, n) (the first CTA), n up to kCollect: bitonic, the part behind n filled up with the largest key.
__device__ __forceinline__ void sort_list(Shared& s, int n) {
  int size = 64;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) s.list[i] = ~uint64_t(0);
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;  // bit j of a is 0
        const uint64_t x = s.list[a], y = s.list[b];
        if ((x > y) == ((a & k) == 0)) {
          s.list[a] = y;
          s.list[b] = x;
        }
      }
      // (pairs up to 32 apart stay within a warp's 64 places)
      if (j > 32 || (j == 1 && k >= 64)) __syncthreads();
      else __syncwarp();
    }
  }
  __syncthreads();
}

// The token out of the collected candidates (the first CTA).
__device__ __forceinline__ void finish(const Params& P, Shared& s, const Row& r, const Weight& w, float per_bin, int64_t row,
                                       uint32_t candidates) {
  const int n = static_cast<int>(s.collected);
  sort_list(s, n);
  const uint64_t least_w = r.min_p > 0.f ? w.part_up(r.min_p) : 0;
  const uint32_t most = r.top_k > 0 ? static_cast<uint32_t>(r.top_k) : 0xffffffffu;
  const int per = (n + kThreads - 1) / kThreads, e0 = threadIdx.x * per, e1 = min(e0 + per, n);
  const uint64_t seg[4] = {s.segment[0], s.segment[1], s.segment[2], s.segment[3]};
  // a candidate's interval, from its bin
  const auto interval = [&](float x) {
    const int b = min(static_cast<int>((w.top - x) * per_bin), kBins - 1);
    return (s.plan.count > 1 && b >= s.plan.begin[1]) + (s.plan.count > 2 && b >= s.plan.begin[2]);
  };
  const auto before = [&](int j) { return seg[0] + (j > 0 ? seg[1] : 0) + (j > 1 ? seg[2] : 0); };
  uint64_t mine = 0, kept = 0, all;
  for (int e = e0; e < e1; ++e) {
    const float x = logit_of(s.list[e]);
    const uint64_t m = w.of(x, s.table);
    mine += m;
    if (m >= least_w && static_cast<uint32_t>(s.plan.rank[interval(x)] + e) < most) kept += m;
  }
  const uint64_t first = block_scan(mine, s, &all) - mine;  // of this thread's part
  const uint64_t z1 = block_sum(kept, s) + seg[0] + seg[1] + seg[2] + seg[3];
  // p z1, in 128 bits
  const uint64_t share = fraction64(r.top_p), p_hi = __umul64hi(z1, share), p_lo = z1 * share;
  const auto is_kept = [&](int e, float x, uint64_t m, uint64_t upto) {
    const uint32_t rank = static_cast<uint32_t>(s.plan.rank[interval(x)] + e);
    return rank < most && m >= least_w && (r.top_p >= 1.f || rank == 0 || upto < p_hi || (upto == p_hi && p_lo != 0));
  };
  uint64_t z2 = z1;
  if (r.top_p < 1.f) {
    uint64_t at = first, top = 0;
    for (int e = e0; e < e1; ++e) {
      const float x = logit_of(s.list[e]);
      const uint64_t m = w.of(x, s.table), upto = before(interval(x)) + at;
      if (is_kept(e, x, m, upto)) top = upto + m;
      at += m;
    }
    z2 = ~block_min(~top, s);
  }
  const uint64_t target = part_of(z2, r.u);
  uint64_t at = first, token = ~uint64_t(0);
  for (int e = e0; e < e1; ++e) {
    const float x = logit_of(s.list[e]);
    const uint64_t m = w.of(x, s.table);
    at += m;
    if (before(interval(x)) + at > target) {
      token = e;
      break;
    }
  }
  token = block_min(token, s);
  if (threadIdx.x == 0) {
    const uint64_t key = s.list[min(token, static_cast<uint64_t>(n - 1))];
    P.tokens[row] = static_cast<int32_t>(key & 0xffffffffu);
    if (P.logprobs) P.logprobs[row] = w.log_share(logit_of(key), s.table, z2);
  }
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
    s.sum[0] = s.sum[1] = s.most = 0;
    s.least = ~0ull;
  }
  __syncthreads();
  n = warp_sum(n);
  m = warp_sum(m);
  lo = warp_min(lo);
  hi = ~warp_min(~hi);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&s.sum[0], static_cast<unsigned long long>(n));
    atomicAdd(&s.sum[1], static_cast<unsigned long long>(m));
    atomicMin(&s.least, static_cast<unsigned long long>(lo));
    atomicMax(&s.most, static_cast<unsigned long long>(hi));
  }
  cluster.sync();
  *count = *mass = *most = 0;
  *least = ~uint64_t(0);
  for (int c = 0; c < kCtas; ++c) {
    const Shared* o = cluster.map_shared_rank(&s, c);
    *count += o->sum[0];
    *mass += o->sum[1];
    *least = min(*least, static_cast<uint64_t>(o->least));
    *most = max(*most, static_cast<uint64_t>(o->most));
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
__device__ __noinline__ void by_bisection(const Params& P, Shared& s, const Row& r, const Weight& w, int64_t row, int rank,
                                          uint32_t candidates) {
  const uint64_t all = ~uint64_t(0);
  uint64_t end = all, count, mass, x, y;
  if (r.top_k > 0 && static_cast<uint32_t>(r.top_k) < candidates)
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
    if (P.logprobs) P.logprobs[row] = w.log_share(logit_of(key), s.table, mass);
  }
}

// ------------------------------------------------------------------ kernel
template <typename T, int kCtas>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) sample_kernel(const Params P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = kCtas == 1 ? 0 : static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / kCtas;
  const int first = rank * kThreads + threadIdx.x, step = kCtas * kThreads;
  if (threadIdx.x < 256) s.table[threadIdx.x] = kPowers.v[threadIdx.x];
  for (int b = threadIdx.x; b < kBins; b += kThreads) s.bins[b] = 0;
  grid_dep_wait();
  grid_dep_launch();
  Row r;
  r.temperature = P.temperature ? __ldg(P.temperature + row) : 1.f;
  r.top_p = P.top_p ? __ldg(P.top_p + row) : 1.f;
  r.min_p = P.min_p ? __ldg(P.min_p + row) : 0.f;
  r.top_k = P.top_k ? __ldg(P.top_k + row) : 0;
  r.u = __ldg(P.uniform + row);
  // the largest logit
  float top = -INFINITY;
  int32_t at = 0;
  uint32_t finite = 0;
  each<T>(P, row, first, step, [&](float x, int i) {
    if (!candidate(x)) return;
    ++finite;
    if (x > top) {
      top = x;
      at = i;
    }
  });
  const uint64_t best = block_min(finite > 0 ? key_of(top, at) : ~uint64_t(0), s), here = block_sum(finite, s);
  if (threadIdx.x < kCtas) {
    Shared* o = cluster.map_shared_rank(&s, threadIdx.x);
    o->best[rank] = best;
    o->finite[rank] = here;
  }
  cluster.sync();
  uint64_t key = ~uint64_t(0);
  uint32_t candidates = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    key = min(key, static_cast<uint64_t>(s.best[c]));
    candidates += static_cast<uint32_t>(s.finite[c]);
  }
  const bool wrong = !(r.temperature >= 0.f && r.temperature <= 3.4e38f) || !(r.u >= 0.f && r.u < 1.f) || !(r.top_p >= 0.f) ||
                     !(r.min_p <= 1.f);
  if (wrong || candidates == 0 || r.temperature == 0.f) {
    if (rank == 0 && threadIdx.x == 0) {
      const bool none = wrong || candidates == 0;
      if (wrong) flag_error(P.err, kErrSetting);
      P.tokens[row] = none ? -1 : static_cast<int32_t>(key & 0xffffffffu);
      if (P.logprobs) P.logprobs[row] = none ? -INFINITY : 0.f;
    }
    return;
  }
  const Weight w(logit_of(key), r.temperature, P.shift);
  const float per_bin = fminf(w.ch * kBinsPerUnit, 3.0e38f);
  // how many fall into each bin
  each<T>(P, row, first, step, [&](float x, int) {
    if (!candidate(x)) return;
    const float y = (w.top - x) * per_bin;
    if (y < kBins - 1.f) atomicAdd(&s.bins[static_cast<int>(y)], 1u);
  });
  cluster.sync();
  Shared* head = cluster.map_shared_rank(&s, 0);
  for (int b = rank * (kBins / kCtas) + threadIdx.x; b < (rank + 1) * (kBins / kCtas); b += kThreads) {
    uint32_t n = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) n += cluster.map_shared_rank(&s, c)->bins[b];
    head->total[b] = n;
  }
  cluster.sync();
  if (rank == 0) {
    // the rest are in the last bin
    uint64_t counted = 0;
    for (int b = threadIdx.x; b < kBins - 1; b += kThreads) counted += s.total[b];
    counted = block_sum(counted, s);
    if (threadIdx.x == 0) s.total[kBins - 1] = candidates - static_cast<uint32_t>(counted);
    __syncthreads();
    make_plan(s, r, candidates);
  }
  cluster.sync();
  if (rank != 0 && threadIdx.x < sizeof(Plan) / 4)
    reinterpret_cast<int32_t*>(&s.plan)[threadIdx.x] = reinterpret_cast<const int32_t*>(&head->plan)[threadIdx.x];
  __syncthreads();
  for (int b = threadIdx.x; b < kBins; b += kThreads) {
    int kind = b > s.plan.last ? kIgnore : 0;
    for (int j = 0; j < s.plan.count; ++j) {
      if (b >= s.plan.begin[j] && b <= s.plan.end[j]) kind = kGather;
      else if (kind < kIgnore && b > s.plan.end[j]) ++kind;
    }
    s.kind[b] = static_cast<uint8_t>(kind);
  }
  __syncthreads();
  // candidates of the borders' bins are collected, the others' weights summed up
  uint64_t mass[4] = {0, 0, 0, 0};
  each<T>(P, row, first, step, [&](float x, int i) {
    if (!candidate(x)) return;
    const int kind = s.kind[static_cast<int>(fminf((w.top - x) * per_bin, kBins - 1.f))];
    if (kind == kIgnore) return;
    if (kind == kGather) {
      const uint32_t place = atomicAdd(&head->collected, 1u);
      if (place < kCollect) head->list[place] = key_of(x, i);
      return;
    }
    const uint64_t m = w.of(x, s.table);
#pragma unroll
    for (int k = 0; k < 4; ++k) mass[k] += kind == k ? m : 0;
  });
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t m = warp_sum(mass[k]);
    if ((threadIdx.x & 31) == 0 && m) atomicAdd(&head->segment[k], static_cast<unsigned long long>(m));
  }
  cluster.sync();
  const bool many = head->collected > kCollect;
  cluster.sync();  // (the first CTA's memory has been read)
  if (many) by_bisection<T, kCtas>(P, s, r, w, row, rank, candidates);
  else if (rank == 0) finish(P, s, r, w, per_bin, row, candidates);
}

template <typename T, int kCtas>
int launch(const Params& p, int32_t rows, cudaStream_t s) {
  static uint64_t smem_set = 0;
  const int st = set_smem_once(reinterpret_cast<const void*>(sample_kernel<T, kCtas>), sizeof(Shared), &smem_set);
  return st ? st : cuda_status(launch_k(sample_kernel<T, kCtas>, dim3(rows * kCtas), dim3(kThreads), sizeof(Shared), s, p));
}

template <typename T>
int launch_rows(const Params& p, int32_t rows, int num_sms, cudaStream_t s) {
  // CTAs a row: as many as the SMs hold two of each, none with less than 1024 logits
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
