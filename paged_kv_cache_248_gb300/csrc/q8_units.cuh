// q8_units.cuh -- what the kernels of the 8-bit attention share: how its work is cut.
//
// A unit is (request, kv head, 2^unit_q_log2 consecutive tokens of the request); it goes over the key tiles (128
// keys) that its last token sees.  All units' key tiles, one after the other, and unit_cost places more for each unit's
// beginning and end, are cut into equal runs, one a CTA, so that one long request and a thousand short ones keep
// every SM equally busy; a CTA derives its run from the lengths by itself, in closed form, without a planning
// launch.  A unit that lies within one run is finished there; of one that is cut, each run leaves its
// rows' unnormalised accumulator, reference and sum, joined by the merge kernel (tree_merge.cuh).
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "pkv_internal.cuh"
#include "tree_merge.cuh"

namespace pkv {

constexpr int kBlocksPerTile = kTileKeys / kBlock;
constexpr int kItemRing = 4;  // items published ahead
constexpr float kLeastV = 8.271806125530277e-25f, kMostV = 1.298074214633707e33f;  // V's scales: 2^-80, 2^110

struct Q8Params {
  const __nv_bfloat16* q;
  const uint8_t *k_cache, *v_cache;
  const float2* scales;
  const int32_t *bt, *seq_lens, *qsl;
  __nv_bfloat16* out;
  uint32_t* err;
  float* part_o;   // [2 * runs][rows_cap][128]
  float* part_ml;  // [2 * runs][rows_cap][2]
  Cut* cuts;       // [2 * runs]
  int64_t num_blocks, num_tokens;
  int32_t num_seqs, max_blocks, max_q, hkv, hq, group, gp_log2, unit_q_log2, unit_cost, rows_cap, min_run, out_v8;
  int32_t least_q, most_q;  // tokens of the requests that the kernel takes
  int32_t reports;          // it zeroes the rows of those that do not fit
  float scale_log2;
};
int launch_q8_chunks(const Q8Params& p, int ctas, cudaStream_t s);

// A part of a unit: what one run does of it.
struct alignas(16) Item {
  int32_t idx;  // -1: the run is over
  int32_t seq, head, slot;  // slot: where its partial goes, -1: the unit is finished here
  int32_t t0, ctx, len, j0;
  int32_t nq, kt0, nt, pad;
};

template <int kThreads>
struct Run {
  int64_t begin, end, base, len;  // places; the first place of the request it begins in; of every run
  int32_t seq;
  int64_t warp_sum[kThreads / 32];
};

// mbar_wait (ptx.cuh) by the SM's clock, which is read in a few cycles; gives up after 2^31 of them,
// about a second.
__device__ __forceinline__ uint32_t sm_clock() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(t));
  return t;
}
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const uint32_t t0 = sm_clock();
  while (!mbar_try_wait(bar, parity))
    if ((abort_flag != nullptr && *abort_flag) || sm_clock() - t0 > 0x7fffffffu) return false;
  return true;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag);
}

__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ __half2 from_e4m3(uint32_t x) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x), __NV_E4M3));
}

// ------------------------------------------------------------------ units
// sum of floor(i / m) over i < x, m = 2^k
__device__ __forceinline__ int64_t floors(int64_t x, int k) {
  const int64_t q = x >> k;
  return ((q * (q - 1) / 2) << k) + q * (x - (q << k));
}

struct Request {
  int32_t t0, q_len, len, units;
  bool wrong;         // to be reported, its rows to zero
  int64_t head_cost;  // of its units of one kv head: a unit costs its key tiles and P.unit_cost

  // Key tiles of unit u.
  __device__ __forceinline__ int32_t tiles(const Q8Params& P, int u) const {
    const int64_t end = static_cast<int64_t>(u + 1) << P.unit_q_log2;
    const int32_t seen = len - q_len + static_cast<int32_t>(end < q_len ? end : q_len);
    return (seen - 1) / kTileKeys + 1;
  }
  // Places of the units before unit u <= units - 1, all of which have Q = 2^unit_q_log2 tokens: unit v - 1 has
  // ceil((ctx + v Q) / 128) tiles, which is floor((a + v) / (128 / Q)) with a = floor((ctx + 127) / Q) for Q up to 128,
  // ceil(ctx / 128) + v Q / 128 for more; v runs from 1 to u.
  __device__ __forceinline__ int64_t before(const Q8Params& P, int u) const {
    const int k = 7 - P.unit_q_log2;
    const int64_t ctx = len - q_len, n = u;
    int64_t tiles;
    if (k >= 0) {
      const int64_t a = (ctx + 127) >> P.unit_q_log2;
      tiles = floors(a + n + 1, k) - floors(a + 1, k);
    } else {
      tiles = n * ((ctx + 127) / 128) + ((n * (n + 1) / 2) << -k);
    }
    return tiles + n * P.unit_cost;
  }
};

__device__ __forceinline__ Request make_request(const Q8Params& P, int32_t q0, int32_t q1, int32_t len) {
  Request r;
  const int64_t n = static_cast<int64_t>(q1) - q0;
  const bool real = n >= 0 && q0 >= 0 && q1 <= P.num_tokens, rows = real && n > 0;
  const bool fits = rows && len >= n && len <= kMaxLen && n <= P.max_q &&
                    (static_cast<int64_t>(len) + kBlock - 1) / kBlock <= P.max_blocks;
  // (of rows that are not real, those that exist)
  r.t0 = max(q0, 0);
  r.q_len = static_cast<int32_t>(max(int64_t(0), min(static_cast<int64_t>(q1), P.num_tokens) - r.t0));
  r.len = len;
  r.wrong = !real || (rows && !fits);
  const bool takes = fits && n >= P.least_q && n <= P.most_q;
  r.units = takes ? ((r.q_len - 1) >> P.unit_q_log2) + 1 : 0;
  r.head_cost = takes ? r.before(P, r.units - 1) + r.tiles(P, r.units - 1) + P.unit_cost : 0;
  return r;
}

__device__ __forceinline__ Request load_request(const Q8Params& P, int i) {
  return make_request(P, __ldg(P.qsl + i), __ldg(P.qsl + i + 1), __ldg(P.seq_lens + i));
}

static __device__ __noinline__ void zero_wrong(const Q8Params& P) {
#pragma unroll 1
  for (int i = blockIdx.x; i < P.num_seqs; i += gridDim.x) {
    const Request r = load_request(P, i);
    if (!r.wrong) continue;
    if (threadIdx.x == 0) flag_error(P.err, kErrLength);
    const int64_t vecs = static_cast<int64_t>(r.q_len) * P.hq * 16;
    uint4* dst = reinterpret_cast<uint4*>(P.out) + static_cast<int64_t>(r.t0) * P.hq * 16;
#pragma unroll 1
    for (int64_t v = threadIdx.x; v < vecs; v += blockDim.x) dst[v] = make_uint4(0, 0, 0, 0);
  }
}

// This CTA's run (all threads).
template <int kThreads>
__device__ __forceinline__ void find_run(const Q8Params& P, Run<kThreads>& c) {
  const int per = (P.num_seqs + kThreads - 1) / kThreads;
  const int i0 = min(static_cast<int>(threadIdx.x) * per, P.num_seqs), i1 = min(i0 + per, P.num_seqs);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t mine = 0;
  bool wrong = false;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const Request r = load_request(P, i);
    mine += r.head_cost * P.hkv;
    wrong |= r.wrong;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) c.warp_sum[warp] = incl;
  const bool any_wrong = __syncthreads_or(wrong);
  int64_t first = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) first += c.warp_sum[w];
    total += c.warp_sum[w];
  }
  int64_t len = (total + gridDim.x - 1) / gridDim.x;
  if (len < P.min_run) len = P.min_run;
  const int64_t begin = len * blockIdx.x, end = begin + len < total ? begin + len : total;
  if (threadIdx.x == 0) {
    c.seq = 0;
    c.base = 0;
    c.begin = begin;
    c.end = end;
    c.len = len;
  }
  __syncthreads();
  if (begin >= first && begin < first + mine) {
    int64_t at = first;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int64_t places = load_request(P, i).head_cost * P.hkv;
      if (begin < at + places) {
        c.seq = i;
        c.base = at;
        break;
      }
      at += places;
    }
  }
  if (any_wrong && P.reports) zero_wrong(P);
  __syncthreads();
}

// Walks the items of a run; the whole warp holds it, lane l the lengths of request rb + l.
struct Walk {
  int64_t pos, end, base;
  int i, rb;
  int32_t q0, q1, len;
};

template <int kThreads>
__device__ __forceinline__ Walk start_walk(const Run<kThreads>& r) {
  return Walk{r.begin, r.end, r.base, r.seq, -64, 0, 0, 0};
}

// The next item (idx -1: none is left).
__device__ __forceinline__ Item next_item(const Q8Params& P, Walk& k, int64_t run_len) {
  Item info{};
  info.idx = -1;
  while (k.pos < k.end) {
    if (k.i - k.rb >= 32) {
      k.rb = k.i;
      const int r = min(k.rb + static_cast<int>(threadIdx.x & 31), P.num_seqs - 1);
      k.q0 = __ldg(P.qsl + r);
      k.q1 = __ldg(P.qsl + r + 1);
      k.len = __ldg(P.seq_lens + r);
    }
    const int src = k.i - k.rb;
    const Request rq = make_request(P, __shfl_sync(0xffffffffu, k.q0, src), __shfl_sync(0xffffffffu, k.q1, src),
                                    __shfl_sync(0xffffffffu, k.len, src));
    const int64_t all = rq.head_cost * P.hkv;
    if (k.pos >= k.base + all) {  // (0 among them)
      k.base += all;
      if (++k.i >= P.num_seqs) k.pos = k.end;  // (lengths that changed meanwhile)
      continue;
    }
    const int64_t off = k.pos - k.base;
    const int head = static_cast<int>(off / rq.head_cost);
    const int64_t in_head = off - head * rq.head_cost;
    int u = 0;  // the last unit that begins at in_head or before
    for (int hi = rq.units - 1; u < hi;) {
      const int mid = u + (hi - u + 1) / 2;
      if (rq.before(P, mid) <= in_head) u = mid;
      else hi = mid - 1;
    }
    // a unit's first unit_cost places stand for its beginning and end, its tiles come after
    const int64_t at = in_head - rq.before(P, u), left = k.end - k.pos;
    const int32_t tiles = rq.tiles(P, u), places = tiles + P.unit_cost;
    const int32_t stop = left < places - at ? static_cast<int32_t>(at + left) : places;
    const int32_t first = max(0, static_cast<int32_t>(at) - P.unit_cost), nt = max(0, stop - P.unit_cost) - first;
    k.pos += stop - at;
    if (nt == 0) continue;
    info.idx = 0;
    info.seq = k.i;
    info.head = head;
    info.t0 = rq.t0;
    info.len = rq.len;
    info.ctx = rq.len - rq.q_len;
    info.j0 = u << P.unit_q_log2;
    info.nq = min(1 << P.unit_q_log2, rq.q_len - info.j0);
    info.kt0 = first;
    info.nt = nt;
    info.slot = nt == tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (first == 0 ? 1 : 0);
    if (info.slot >= 0 && (threadIdx.x & 31) == 0) {  // the runs before that have a part of the unit, and after
      const int64_t before = (first + run_len - 1) / run_len, after = (places - stop + run_len - 1) / run_len;
      P.cuts[info.slot] = Cut{static_cast<int32_t>(before + 1 + after), static_cast<int32_t>(before), info.t0, head,
                              {info.j0, 0}, {info.nq, 0}};
    }
    break;
  }
  return info;
}

}  // namespace pkv
