// k_tree_tc.cu -- attention of drafted trees over the paged cache on tcgen05 tensor cores
// (bf16, head_dim 128).
//
// Mathematics.  Node j of request i sees the keys u < c_i = seq_len - q_len, and of the draft
// the keys c_i + b whose bit b its mask row has; out = sum_u softmax_u(scale q.K_u) V_u over
// those keys, in one pass over the keys with a running maximum and sum per row (fp32) and P
// rounded to bf16 for the second product (one rounding of each weight, half a step of 2^-8
// of it; the row sum takes the weights unrounded).
//
// Rows.  The G query heads of a kv head are folded into the 128 rows of an MMA tile: R = 128 / GP
// nodes x GP heads (GP = G rounded up to a power of two).  A unit is (request, kv head, one
// row tile, or two) and goes over all of the request's key tiles of 128 keys.
//
// Cut.  All units' key tiles, one after the other (and two places more for each unit, whose
// beginning and end take time too: 33 requests of 0..1500 keys 36.2, 31.4, 30.2 us with 0, 1, 2 of
// them), are cut into equal runs, so that one long request and a thousand short ones keep every SM equally busy; a CTA
// derives its runs from the lengths by itself, without a planning launch.  A unit that lies within
// one run is finished there; of one that is cut, each run leaves its rows' unnormalised accumulator,
// maximum and sum, and the merge kernel joins them in order.  A run leaves at most two such
// partials.  Where every kv head of every request that has rows has the same number of units, above
// one, as many runs at a time go through the same keys, each for one of the units, so that K and V come
// from HBM once and not once a unit (8 requests of 32768 keys with 512 rows: 2.17 GB read and 398 us
// one unit after the other, 1.09 GB and 373 us side by side); see side_by_side for what it costs.
//
// Streams.  Two S/P/O accumulator sets live in TMEM, each with a softmax warpgroup of its own, so
// that one softmax runs while the tensor core works for the other.
//   tree_kernel<false>: a stream has a run of its own, of units of one row tile; the streams
//     take turns at the tensor core and at the rings, a tile each, and one's last rows are
//     stored while the other goes on (requests of few rows, or few keys).
//   tree_kernel<true>: a CTA has one run, of units of two row tiles; a stream is a row tile,
//     and every key tile is loaded once for both.
//
// Per CTA (352 threads): warp 0 finds the runs' units and loads Q and K, warp 10 loads V (TMA
// boxes of the blocks' 16-token rows, 128-byte swizzle; 2 K and 2 V tiles in flight: a third V tile
// takes the shared memory that the L1 then lacks, and 5 % more time for the 64 requests below; L2 is
// told to drop what it passed on first, 101.5 us instead of 111 for them), warp 1 issues the MMAs,
// warps 2-5 and 6-9 are the streams' softmax.  The tiles
// that hold drafted keys (the last one or two of a request) take their visibility from the
// mask row's bits, the others see every key.  Their V rows are looked through for values that
// are not finite: a zero weight times those would reach rows that do not see them, so they
// are taken out of the tile and given back, at the end, to the rows that do.
//
// Bound, 32 / 8 heads: 64 requests of 128..4096 keys with 16 nodes read 558 MB: 103 us, of which the
// merge is 7 (82 us at a copy's rate; DRAM 73 % busy).  8 requests of 32768 keys with 64 nodes,
// 64 / 8 heads, are 550 GFLOP: 375 to 425 us as the power limit has it (290 us at the rate of a large
// matrix product, 320 us at the one that the limit sustains); softmax and MMAs of the two streams
// alternate, about 1900 cycles a turn each, and the tensor pipe is busy for 64 % of the time.  One
// request of 500 keys: 10 us, nearly all latency: 1.3 us until its run is known, 2 until its first tile
// is on its way, 0.6 until that is there, 3 for the products and the softmax, 2 for the merge.
//
// All waits are bounded (ptx.cuh).
#include "ptx.cuh"
#include "pkv_internal.cuh"
#include "softmax_row.cuh"
#include "tree_merge.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 352;
constexpr int kKStages = 2;
constexpr int kVStages = 2;
constexpr int kHalfBytes = 16384;
constexpr int kTileBytes = 2 * kHalfBytes;  // 128 x 128 bf16 in two 64-column halves
constexpr int kRing = 4;                    // items published ahead, per ring
constexpr uint32_t kTmemCols = 512;         // S_0, S_1 (P over their first 64 columns), O_0, O_1
constexpr uint32_t kOCol = 256;
constexpr int kBlocksPerTile = kTileKeys / kBlock;
constexpr int kShortKeys = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled when a row's maximum grows by > 2^8

// A part of a unit: what one run does of it.
struct alignas(16) Item {
  int32_t idx;  // -1: the run is over
  int32_t seq, head, slot;  // slot: where its partial goes, -1: the unit is finished here
  int32_t t0, q_len, ctx, len;
  int32_t kt0, nt, pad0, pad1;  // key tiles kt0 .. kt0 + nt - 1
  int32_t j0[2], nq[2];         // row tile w: its first node and how many
};

struct Run {
  int64_t begin, end, base;  // places; the first place of the request it begins in
  int32_t seq;
  int32_t unit;  // of each kv head, -1: all units, one after the other (see "Cut")
};

struct Ctl {
  uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages];
  uint64_t s_full[2], o_full[2], o_free[2], p_full[2][2], q_full[2], q_free[2];
  uint64_t item_full[2][kRing], item_empty[2][kRing];  // one ring per run
  uint64_t drain;
  Item ring[2][kRing];
  int bad[2][kRing];     // a block id outside of the pool
  int spoilt[2][kRing];  // a drafted V row that is not finite
  Run run[2];
  int64_t run_len;
  int64_t warp_sum[kThreads / 32];
  int32_t warp_most[kThreads / 32], warp_least[kThreads / 32];
  uint32_t tmem_base;
  uint32_t q_loads[2];
  uint32_t number[2][8];  // numbers in the rings of a run's latest tiles
  int abort_flag;
};

constexpr int kSmemBytes = (2 + kKStages + kVStages) * kTileBytes + static_cast<int>(sizeof(Ctl));
static_assert(kSmemBytes <= 232448, "tree attention shared memory");

struct Params {
  __nv_bfloat16* out;
  const __nv_bfloat16* v_cache;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* qsl;
  const uint64_t* mask;
  uint32_t* err;
  float* part_o;   // [2 * runs][rows_cap][128]
  float* part_ml;  // [2 * runs][rows_cap][2]
  Cut* cuts;       // [2 * runs]
  int64_t num_blocks, num_tokens;
  int32_t num_seqs, max_blocks, max_q, mask_words;
  int32_t hkv, hq, group, gp, gp_log2, rows_q, unit_q, unit_q_log2, unit_cost, rows_cap, min_run, out_v8;
  int32_t row0[2];  // the MMA tile's row that holds a stream's first row (see launch_tree_tc)
  float scale_log2;
};

// mbar_wait (ptx.cuh) in fewer instructions: this kernel has many waits, and the code that its
// warps run by turns has to stay in the SM's instruction cache (see softmax_warps).  Gives up
// after 2^31 SM cycles, about a second.
__device__ __forceinline__ uint32_t sm_clock() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(t));
  return t;
}
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint32_t t0 = sm_clock();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((abort_flag != nullptr && *abort_flag) || sm_clock() - t0 > 0x7fffffffu) return false;
  }
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_long(smem_u32(bar), parity, abort_flag);
}

__device__ __forceinline__ void raise_abort(Ctl& c, uint32_t* err) {
  *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
  flag_error(err, kErrTimeout);
}

template <typename T>
__device__ __forceinline__ T same(T x) {  // lane 0's value
  return __shfl_sync(0xffffffffu, x, 0);
}

// ------------------------------------------------------------------ units
struct Request {
  int32_t t0, q_len, len;
  bool wrong;            // to be reported, its rows to zero: lengths that do not fit, rows that do not exist
  int32_t tiles, units;  // key tiles of a unit; units of one kv head
  int32_t cost;          // of all its units: a unit costs its key tiles and P.unit_cost

  // Its places where one unit of each kv head counts, or all.
  __device__ __forceinline__ int32_t places(const Params& P, bool one) const {
    return one && cost > 0 ? P.hkv * (tiles + P.unit_cost) : cost;
  }
};

__device__ __forceinline__ Request make_request(const Params& P, int32_t q0, int32_t q1, int32_t len) {
  Request r;
  const int64_t n = static_cast<int64_t>(q1) - q0;
  const bool real = n >= 0 && q0 >= 0 && q1 <= P.num_tokens, rows = real && n > 0;
  bool fits = rows && len >= n && len <= kMaxLen && n <= P.max_q &&
              (static_cast<int64_t>(len) + kBlock - 1) / kBlock <= P.max_blocks;
  // (of rows that are not real, those that exist)
  r.t0 = max(q0, 0);
  r.q_len = static_cast<int32_t>(max(int64_t(0), min(static_cast<int64_t>(q1), P.num_tokens) - r.t0));
  r.len = len;
  r.tiles = static_cast<int>(static_cast<uint32_t>(len - 1) / kTileKeys) + 1;
  r.units = (r.q_len + P.unit_q - 1) >> P.unit_q_log2;
  // (2^31 places and more would be terabytes of K and V, read once a unit)
  const int64_t cost = static_cast<int64_t>(P.hkv) * r.units * (r.tiles + P.unit_cost);
  fits = fits && cost < (int64_t(1) << 31);
  r.wrong = !real || (rows && !fits);
  r.cost = fits ? static_cast<int32_t>(cost) : 0;
  return r;
}

__device__ __noinline__ Request load_request(const Params& P, int i) {
  return make_request(P, __ldg(P.qsl + i), __ldg(P.qsl + i + 1), __ldg(P.seq_lens + i));
}

// Wrong requests are reported and their rows zeroed (by `step` threads, this is number `first`).
__device__ __noinline__ void zero_wrong(const Params& P, int first, int step) {
#pragma unroll 1
  for (int i = blockIdx.x; i < P.num_seqs; i += gridDim.x) {
    const Request r = load_request(P, i);
    if (!r.wrong) continue;
    if (first == 0) flag_error(P.err, kErrLength);
    const int64_t vecs = static_cast<int64_t>(r.q_len) * P.hq * 16;
    uint4* dst = reinterpret_cast<uint4*>(P.out) + static_cast<int64_t>(r.t0) * P.hq * 16;
#pragma unroll 1
    for (int64_t v = first; v < vecs; v += step) dst[v] = make_uint4(0, 0, 0, 0);
  }
}

// Run number k of this CTA: `total` places of one unit of each kv head (units > 0) or of all (0) cut
// into equal runs.
template <int kRuns>
__device__ __forceinline__ Run cut_run(const Params& P, int k, int64_t total, uint32_t units, int64_t* len) {
  uint32_t runs = gridDim.x * kRuns, number = k * gridDim.x + blockIdx.x, unit = 0;
  if (units > 0) {
    runs /= units;
    unit = number / runs;
    number -= unit * runs;
  }
  const int64_t even = total < 0x7fffffff ? (static_cast<uint32_t>(total) + runs - 1) / runs : (total + runs - 1) / runs;
  *len = even > P.min_run ? even : P.min_run;
  Run r;
  r.begin = *len * number;
  r.end = r.begin + *len < total ? r.begin + *len : total;
  if (units > 0 && unit >= units) r.end = r.begin;  // (a CTA too many)
  r.base = 0;
  r.seq = 0;
  r.unit = units > 0 ? static_cast<int32_t>(unit) : -1;
  return r;
}

// Whether so many units of each kv head go side by side.  Every unit gets equally many runs, and the CTAs
// that are left over rest; where those are more than a sixth the units come one after the other.  One
// request of 8000 keys on 152 SMs, side by side / one after the other: 38 units 48.4 / 54.5 us, 70 (12 SMs
// rest) 86.7 / 85.9, 128 (24) 150.0 / 149.2, 60 (32) 82.5 / 73.9, 51 (50) 79.4 / 64.6, 80 (72) 131.9 / 95.7;
// of 2000 keys 128 units 78.9 / 88.9, 60 units 49.1 / 46.3.
__device__ __forceinline__ bool side_by_side(uint32_t units) {
  return units > 1 && 6 * (gridDim.x / units * units) >= 5 * gridDim.x;
}

// This CTA's kRuns runs: run k * CTAs + CTA, so that few runs have an SM each (all threads).
template <int kRuns>
__device__ void find_runs(const Params& P, Ctl& c) {
  const int per = (P.num_seqs + kThreads - 1) / kThreads;
  const int i0 = min(static_cast<int>(threadIdx.x) * per, P.num_seqs), i1 = min(i0 + per, P.num_seqs);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t mine = 0;
  int32_t most = 0, least = 0x7fffffff;  // units of a kv head, of requests that have any
  bool wrong = false;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const Request r = load_request(P, i);
    mine += r.cost;
    wrong |= r.wrong;
    if (r.cost > 0) {
      most = max(most, r.units);
      least = min(least, r.units);
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) {
    c.warp_most[warp] = most;
    c.warp_least[warp] = least;
  }
  const bool any_wrong = __syncthreads_or(wrong);
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    most = max(most, c.warp_most[w]);
    least = min(least, c.warp_least[w]);
  }
  const bool one = kRuns == 1 && most == least && side_by_side(most);
  if (one) mine /= most;
  int64_t incl = mine;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) c.warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += c.warp_sum[w];
    total += c.warp_sum[w];
  }
  Run run[kRuns];
  int64_t len;
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    run[k] = cut_run<kRuns>(P, k, total, one ? most : 0, &len);
    if (threadIdx.x == 0) c.run[k] = run[k];
  }
  if (threadIdx.x == 0) c.run_len = len;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    const int64_t begin = run[k].begin;
    if (begin >= before && begin < before + mine) {
      int64_t at = before;
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        const int64_t places = load_request(P, i).places(P, one);
        if (begin < at + places) {
          c.run[k].seq = i;
          c.run[k].base = at;
          break;
        }
        at += places;
      }
    }
  }
  if (any_wrong) zero_wrong(P, threadIdx.x, kThreads);
  __syncthreads();
}

// The same for up to kFewSeqs requests by warp 0 alone, which is the one that walks the runs: no
// barriers, and the requests' loads are all on their way at once (one request 9.8 instead of 10.9
// us, 33 requests 30.2 instead of 31.4, 64 requests 101.5 instead of 102.3).
constexpr int kFewSeqs = 128;
template <int kRuns>
__device__ void find_runs_few(const Params& P, Ctl& c) {
  constexpr int kSets = kFewSeqs / 32;
  const int lane = threadIdx.x & 31;
  int32_t q0[kSets], q1[kSets], len[kSets];
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int i = 32 * s + lane;
    q0[s] = q1[s] = len[s] = 0;
    if (i < P.num_seqs) {
      q0[s] = __ldg(P.qsl + i);
      q1[s] = __ldg(P.qsl + i + 1);
      len[s] = __ldg(P.seq_lens + i);
    }
  }
  int64_t total = 0, before[kSets];
  int32_t cost[kSets];
  bool wrong = false;
  int32_t most = 0, least = 0x7fffffff;  // units of a kv head, of requests that have any
  Request r[kSets];
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    r[s].cost = 0;
    if (32 * s < P.num_seqs) {
      r[s] = make_request(P, q0[s], q1[s], len[s]);
      wrong |= r[s].wrong;
      if (r[s].cost > 0) {
        most = max(most, r[s].units);
        least = min(least, r[s].units);
      }
    }
  }
  const int32_t units = kRuns == 1 ? __reduce_max_sync(0xffffffffu, most) : 0;
  const bool one = kRuns == 1 && units == __reduce_min_sync(0xffffffffu, least) && side_by_side(units);
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    before[s] = cost[s] = 0;
    if (32 * s < P.num_seqs) {
      cost[s] = r[s].places(P, one);
      int64_t incl = cost[s];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      before[s] = total + incl - cost[s];
      total += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    int64_t places;
    const Run run = cut_run<kRuns>(P, k, total, one ? units : 0, &places);
    if (lane == 0) {
      c.run[k] = run;
      c.run_len = places;
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      if (run.begin >= before[s] && run.begin < before[s] + cost[s]) {
        c.run[k].seq = 32 * s + lane;
        c.run[k].base = before[s];
      }
    }
  }
  if (__any_sync(0xffffffffu, wrong)) zero_wrong(P, lane, 32);
  __syncwarp();
}

// Walks the items of a run; the whole warp holds it, lane l the lengths of request rb + l.
struct Walk {
  int64_t pos, end, base;
  int i, unit, rb;
  int32_t q0, q1, len;
};

__device__ __forceinline__ Walk start_walk(const Run& r) {
  return Walk{r.begin, r.end, r.base, r.seq, r.unit, -64, 0, 0, 0};
}

// The next item of run number `run` (idx -1: none is left).
__device__ __forceinline__ Item next_item(const Params& P, Walk& k, int run, int64_t run_len) {
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
    const int32_t all = rq.places(P, k.unit >= 0);
    if (k.pos >= k.base + all) {  // (0 among them)
      k.base += all;
      if (++k.i >= P.num_seqs) k.pos = k.end;  // (lengths that changed meanwhile)
      continue;
    }
    // a unit's first unit_cost places stand for its beginning and end, its tiles come after
    const uint32_t off = static_cast<uint32_t>(k.pos - k.base);
    const uint32_t places = rq.tiles + P.unit_cost;
    int unit = static_cast<int>(off / places);
    const uint32_t at = off - unit * places;
    if (k.unit >= 0) unit = unit * rq.units + k.unit;
    const int64_t left = k.end - k.pos;  // this run's places of the unit: [at, stop)
    const uint32_t stop = left < places - at ? at + static_cast<uint32_t>(left) : places;
    const int first = max(0, static_cast<int>(at) - P.unit_cost);
    const int nt = max(0, static_cast<int>(stop) - P.unit_cost) - first;
    k.pos += stop - at;
    if (nt == 0) continue;
    info.idx = 0;
    info.seq = k.i;
    info.t0 = rq.t0;
    info.q_len = rq.q_len;
    info.len = rq.len;
    info.ctx = rq.len - rq.q_len;
    info.kt0 = first;
    info.nt = nt;
    info.head = static_cast<int>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(rq.units));
    const int j = (unit - info.head * rq.units) << P.unit_q_log2;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      info.j0[w] = j + w * P.rows_q;
      info.nq[w] = max(0, min(P.rows_q, min(rq.q_len, j + P.unit_q) - info.j0[w]));
    }
    info.slot = info.nt == rq.tiles ? -1 : 2 * run + (first == 0 ? 1 : 0);
    if (info.slot >= 0 && (threadIdx.x & 31) == 0) {  // the runs before that have a part of the unit, and after
      const uint32_t len = run_len < 0x7fffffff ? static_cast<uint32_t>(run_len) : 0x7fffffffu;
      const uint32_t before = (static_cast<uint32_t>(first) + len - 1) / len, after = (places - stop + len - 1) / len;
      P.cuts[info.slot] = Cut{static_cast<int32_t>(before + 1 + after), static_cast<int32_t>(before), info.t0, info.head,
                              {info.j0[0], info.j0[1]}, {info.nq[0], info.nq[1]}};
    }
    break;
  }
  return info;
}

// ------------------------------------------------------------------ loads
// Publishes an item in ring k (the whole warp).
__device__ __forceinline__ bool publish(Ctl& c, int k, uint32_t it, const Item& info, volatile int* abort_flag) {
  const int slot = it % kRing;
  if (!wait_for(&c.item_empty[k][slot], ((it / kRing) & 1) ^ 1, abort_flag)) return false;
  if ((threadIdx.x & 31) == 0) {
    c.ring[k][slot] = info;
    c.bad[k][slot] = 0;
    c.spoilt[k][slot] = 0;
    mbar_arrive(&c.item_full[k][slot]);
  }
  __syncwarp();
  return true;
}

// Q tile w: the item's rows from node j0 on.
__device__ __forceinline__ bool load_q(const Params& P, const CUtensorMap* qmap, Ctl& c, uint8_t* qbuf, int w,
                                       const Item& info, int j0, volatile int* abort_flag) {
  const uint32_t n = c.q_loads[w];
  if (!wait_for(&c.q_free[w], (n & 1) ^ 1, abort_flag)) return false;
  if ((threadIdx.x & 31) == 0) {
    uint8_t* q = qbuf + w * kTileBytes;
    mbar_arrive_expect_tx(&c.q_full[w], kTileBytes);
    const int32_t y = info.head * P.group, z = info.t0 + j0;
    tma_load_3d(q, qmap, &c.q_full[w], 0, y, z, l2_policy_evict_first());
    tma_load_3d(q + kHalfBytes, qmap, &c.q_full[w], 64, y, z, l2_policy_evict_first());
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) c.q_loads[w] = n + 1;
  __syncwarp();
  return true;
}

// A run's item as a producer goes through it, and this lane's block id of its next tile (lanes 0-7).
struct Tiles {
  int32_t seq, head, len;
  int32_t tile, end;  // the next tile and the item's end
  int32_t id;
  uint32_t it, tiles;  // items and tiles of the run so far
  int32_t live;

  __device__ __forceinline__ void load_id(const Params& P) {
    const int lane = threadIdx.x & 31, at = tile * kBlocksPerTile + lane;
    id = lane < kBlocksPerTile && at <= (len - 1) / kBlock ? __ldg(P.bt + static_cast<int64_t>(seq) * P.max_blocks + at) : 0;
  }
};

// With two runs, a turn works on `a` and the two states change places after it.
template <typename T>
__device__ __forceinline__ void change_places(T& a, T& b) {
  const T t = a;
  a = b;
  b = t;
}

// The producers walk the runs' tiles in the order in which the MMA thread takes them: a tile
// of each run by turns (one run: its tiles).  The K producer finds the items, publishes them
// and loads Q too; the V producer reads the items like the other warps.  Both run this one
// piece of code, to keep it small.
template <int kRuns>
__device__ void producer_warp(const Params& P, bool is_k, const CUtensorMap* qmap, const CUtensorMap* map, Ctl& c,
                              uint8_t* qbuf, uint8_t* buf) {
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &c.abort_flag;
  uint64_t* full = is_k ? c.kfull : c.vfull;
  uint64_t* empty = is_k ? c.kempty : c.vempty;
  const int stages = is_k ? kKStages : kVStages;
  Walk walk[kRuns];  // (K)
  if (is_k) {
#pragma unroll 1
    for (int k = 0; k < kRuns; ++k) walk[k] = start_walk(c.run[k]);
    if (lane < 2 * kRuns) P.cuts[2 * ((lane >> 1) * gridDim.x + blockIdx.x) + (lane & 1)].parts = 0;
    __syncwarp();
  }
  Tiles a{0, 0, 1, 0, 0, 0, 0, 0, 1}, b = a;
  uint32_t n = 0;
  int live = kRuns, s = 0, phase = 1;  // of the next slot
  bool ok = true;
#pragma unroll 1
  for (int k = 0; ok && live > 0; k ^= kRuns - 1) {
    if (a.live && a.tile == a.end) {
      const int slot = a.it % kRing;
      Item item;
      if (is_k) {
        item = next_item(P, walk[k], k * gridDim.x + blockIdx.x, c.run_len);
      } else {
        ok = wait_for(&c.item_full[k][slot], (a.it / kRing) & 1, abort_flag);
        if (!ok) break;
        item = c.ring[k][slot];
        __syncwarp();
      }
      a.live = item.idx >= 0;
      a.seq = item.seq;
      a.head = item.head;
      a.len = item.len;
      a.tile = item.kt0;
      a.end = item.kt0 + item.nt;
      if (a.live) a.load_id(P);
      else --live;
      if (is_k) {
        ok = publish(c, k, a.it, item, abort_flag);
#pragma unroll 1
        for (int w = 0; w < 3 - kRuns && ok && a.live; ++w)  // the item's one row tile, or two
          if (kRuns == 2 || item.nq[w] > 0)
            ok = load_q(P, qmap, c, qbuf, kRuns == 2 ? k : w, item, (w ? item.j0[1] : item.j0[0]) - (P.row0[k] >> P.gp_log2),
                        abort_flag);
        if (!ok) break;
      } else if (a.live && lane == 0) {
        mbar_arrive(&c.item_empty[k][slot]);
      }
      ++a.it;
    }
    if (a.live) {
      const int tile = a.tile;
      int cur = a.id;
      if (++a.tile < a.end) a.load_id(P);  // loads while this tile waits for its slot
      const bool wrong = cur < 0 || cur >= P.num_blocks;
      if (wrong) cur = 0;
      if (is_k) {
        if (__any_sync(0xffffffffu, wrong)) {
          if (wrong) flag_error(P.err, kErrBlockId);
          if (lane == 0) c.bad[k][(a.it - 1) % kRing] = 1;
          __syncwarp();
        }
        if (lane == 0) c.number[k][a.tiles % 8] = n;
        ++a.tiles;
      }
      // K or V of the tile into its ring slot: 2 boxes of 16 rows per block
      const int nblk = min(kBlocksPerTile, (a.len - 1) / kBlock + 1 - tile * kBlocksPerTile);
      const int32_t row = (cur * P.hkv + a.head) * kBlock;
      ok = wait_for(&empty[s], phase, abort_flag);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(nblk) * 4096u);
      __syncwarp();
      if (lane < nblk) {
        uint8_t* d = buf + s * kTileBytes + lane * 2048;
        tma_load_2d(d, map, &full[s], 0, row, l2_policy_evict_first());
        tma_load_2d(d + kHalfBytes, map, &full[s], 64, row, l2_policy_evict_first());
      }
      ++n;
      if (++s == stages) {
        s = 0;
        phase ^= 1;
      }
    }
    if (kRuns == 2) change_places(a, b);
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
  if (*abort_flag) {  // copies already issued land before the CTA's shared memory goes away
#pragma unroll 1
    for (uint32_t i = n > static_cast<uint32_t>(stages) ? n - stages : 0; i < n; ++i)
      wait_for(&full[i % stages], (i / stages) & 1, nullptr);
#pragma unroll 1
    for (int w = 0; w < 2 && is_k; ++w) {
      const uint32_t q = c.q_loads[w];
      if (q > 0) wait_for(&c.q_full[w], (q - 1) & 1, nullptr);
    }
  }
}

// ------------------------------------------------------------------ MMA warp
// One elected thread issues every MMA, but the whole warp walks through the tiles, with values
// that the compiler can tell to be the same in all of its lanes: the operands of an MMA live in
// uniform registers, and values of one thread have to be moved there before each (a tenth
// more time for 8 requests of 32768 keys).
// A stream's step is P V of its tile before, then S of its next tile: MMAs of one thread complete in
// order, so S cannot overwrite the P that this P V reads, and S being complete tells the softmax
// that O holds every tile before.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
struct Issuer {
  Ctl& c;
  uint32_t tmem, q, k, v;  // shared-memory addresses of the Q tiles and the rings
  volatile int* abort_flag;
  uint32_t p_phase, o_phase, q_phase;  // bit w: the phase to wait for next
  bool issued, failed;

  // A wait that is given up may be given up by some lanes only, and elect.sync wants them all: so the
  // turn goes on, on whatever is there, and the warp votes at its end (well-defined, if useless: the
  // operands are this CTA's memory, and the call reports the timeout).
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) { failed |= !wait_for(bar, parity, abort_flag); }
  __device__ __forceinline__ bool ok() { return !__any_sync(0xffffffffu, failed); }

  // O_w += P_w V of the tile in V slot `slot`; `first` begins O_w anew, `last` reports it.
  // (P being there means that V is: the softmax waits for it and looks through it.)
  __device__ __forceinline__ void pv(int w, uint32_t slot, bool first, bool last) {
    constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false, true);
    const uint64_t b = umma_smem_desc(v + slot * kTileBytes, kHalfBytes, 1024, kLayout128B);
    const uint32_t s_col = tmem + 128 * w;
    wait(&c.p_full[w][0], p_phase >> w & 1);
    if (first) {
      wait(&c.o_free[w], (o_phase >> w & 1) ^ 1);
      o_phase ^= 1u << w;
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      if (hf) wait(&c.p_full[w][1], p_phase >> w & 1);
      tc_fence_after();
      if (elected()) {
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          umma_f16_ts(s_col + kOCol, s_col + 32 * hf + 8 * k4, umma_desc_advance(b, (4 * hf + k4) * 2048), idesc,
                      (!first || hf + k4 > 0) ? 1u : 0u);
        if (hf && last) umma_commit(&c.o_full[w]);
      }
    }
    p_phase ^= 1u << w;
  }

  // S_w = Q_w K^T of the tile in K slot `slot`, whose turn's parity is given; `last`: Q_w has been read.
  __device__ __forceinline__ void s(int w, uint32_t slot, uint32_t parity, bool last) {
    constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false, false);
    wait(&c.kfull[slot], parity);
    tc_fence_after();
    const uint64_t a = umma_smem_desc(q + w * kTileBytes, 16, 1024, kLayout128B);
    const uint64_t b = umma_smem_desc(k + slot * kTileBytes, 16, 1024, kLayout128B);
    if (elected()) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t off = h * kHalfBytes + kk * 32;
          umma_f16_ss(tmem + 128 * w, umma_desc_advance(a, off), umma_desc_advance(b, off), idesc, h + kk > 0);
        }
      }
      umma_commit(&c.s_full[w]);
      if (last) umma_commit(&c.q_free[w]);
    }
    issued = true;
  }

  __device__ __forceinline__ void q_ready(int w) {
    wait(&c.q_full[w], q_phase >> w & 1);
    q_phase ^= 1u << w;
  }
};

template <int kRuns>
__device__ void mma_warp(const Params& P, Ctl& c, uint8_t* qbuf, uint8_t* kbuf, uint8_t* vbuf, uint32_t tmem) {
  static_assert(kKStages == 2 && kVStages == 2, "a tile's slots are its number's lowest bit");
  volatile int* abort_flag = &c.abort_flag;
  Issuer x{c, tmem, smem_u32(qbuf), smem_u32(kbuf), smem_u32(vbuf), abort_flag, 0, 0, 0, false, false};
  uint32_t n = 0;  // tiles
  bool ok = true;
  if (kRuns == 2) {
    struct State {
      uint32_t it, before;
      int nt, j, live, pending;
    };
    State a{0, 0, 0, 0, 1, 0}, b{0, 0, 0, 0, 1, 0};
#pragma unroll 1
    for (int w = 0; ok && (a.live | b.live); w ^= 1) {
      if (a.pending) x.pv(w, a.before, a.j == 1, a.j == a.nt);
      a.pending = 0;
      if (a.live && a.j == a.nt) {
        const int slot = a.it % kRing;
        x.wait(&c.item_full[w][slot], (a.it / kRing) & 1);
        ok = x.ok();
        if (ok) {
          a.nt = same(c.ring[w][slot].nt);
          a.live = same(c.ring[w][slot].idx) >= 0;
          ++a.it;
          a.j = 0;
          if (a.live) {
            if (elected()) mbar_arrive(&c.item_empty[w][slot]);
            x.q_ready(w);
          }
        }
      }
      if (ok && a.live) {
        ++a.j;
        x.s(w, n & 1, n >> 1 & 1, a.j == a.nt);
        a.before = n++ & 1;
        a.pending = 1;
        ok = x.ok();
      }
      change_places(a, b);
    }
  } else {
    uint32_t it = 0;
    while (ok) {
      const int slot = it % kRing;
      x.wait(&c.item_full[0][slot], (it / kRing) & 1);
      ok = x.ok();
      if (!ok) break;
      const int nt = same(c.ring[0][slot].nt), rows = same(c.ring[0][slot].nq[1]) > 0 ? 2 : 1;
      const bool over = same(c.ring[0][slot].idx) < 0;
      ++it;
      if (over) break;
      if (elected()) mbar_arrive(&c.item_empty[0][slot]);
      x.q_ready(0);
      if (rows == 2) x.q_ready(1);
      // turns of the row tiles: 0, 1, 0, 1, ... (one row tile: 0, 0, ...)
      int w = 0;
#pragma unroll 1
      for (int j = 0; j <= nt && ok;) {
        if (j > 0) x.pv(w, (n + j - 1) & 1, j == 1, j == nt);
        if (j < nt) x.s(w, (n + j) & 1, (n + j) >> 1 & 1, j == nt - 1);
        ok = x.ok();
        if (++w == rows) {
          w = 0;
          ++j;
        }
      }
      n += nt;
    }
  }
  if (!ok && !*abort_flag && (threadIdx.x & 31) == 0) raise_abort(c, P.err);
  __syncwarp();
  // every MMA, and the arrivals that its commits trigger, is over before TMEM is freed
  if (x.issued) {
    if (elected()) umma_commit(&c.drain);
    wait_for(&c.drain, 0, nullptr);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax warps
// Bits s .. s + 63 of what a row sees, counted from its first drafted key (s < 0: context,
// seen whole), without those past the draft.
__device__ __noinline__ uint64_t seen_bits(const uint64_t* row, int words, int q_len, int s) {
  if (s <= -64) return ~uint64_t(0);
  if (s >= q_len) return 0;
  uint64_t b;
  if (s < 0) {
    b = (__ldg(row) << -s) | ((uint64_t(1) << -s) - 1);
  } else {
    const int w = s >> 6, sh = s & 63;
    b = __ldg(row + w) >> sh;
    if (sh && w + 1 < words) b |= __ldg(row + w + 1) << (64 - sh);
  }
  const int left = q_len - s;
  return left < 64 ? b & ((uint64_t(1) << left) - 1) : b;
}

// Bits 15 and 31 tell whether a bf16 of the pair is an infinity or NaN (its exponent all ones).
__device__ __forceinline__ uint32_t not_finite2(uint32_t x) { return (x & 0x7f807f80u) + 0x00800080u; }

// The pair with a zero in the place of each infinity or NaN.
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

// Takes what is not finite out of row r of a V tile (all of a row past the context), so that a
// weight of 0 can stand for a key that a row does not see.  Returns whether it took something
// out that a row may see.
__device__ __noinline__ bool clean_v_row(uint8_t* vtile, int r, bool past) {
  // starting each lane at chunk r mod 8 spreads eight lanes over all banks
  uint8_t* row = vtile + r * 128;
  bool spoilt = false;
#pragma unroll 1
  for (int half = 0; half < 2; ++half, row += kHalfBytes) {
    if (past) {
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) *reinterpret_cast<uint4*>(row + ((ch + r) & 7) * 16) = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 x[8];
    uint32_t any = 0;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) x[ch] = *reinterpret_cast<uint4*>(row + ((ch + r) & 7) * 16);
#pragma unroll
    for (int ch = 0; ch < 8; ++ch)
      any |= not_finite2(x[ch].x) | not_finite2(x[ch].y) | not_finite2(x[ch].z) | not_finite2(x[ch].w);
    if (any & 0x80008000u) {
      spoilt = true;
#pragma unroll 1
      for (int ch = 0; ch < 8; ++ch) {
        uint4* at = reinterpret_cast<uint4*>(row + ((ch + r) & 7) * 16);
        const uint4 y = *at;
        *at = make_uint4(finite2(y.x), finite2(y.y), finite2(y.z), finite2(y.w));
      }
    }
  }
  if (past || spoilt) fence_proxy_async_smem();
  return spoilt;
}

// Gives the values that clean_v_row took out of an item's tiles back to a row that sees them, in
// the row's stored result: sums with what is not finite are not finite (rare).
__device__ __noinline__ void give_back(const Params& P, const Item& item, const uint64_t* mrow, int kt0, int nt,
                                       uint8_t* dst) {
  const int b1 = min((kt0 + nt) * kTileKeys, item.len);
  for (int u = max(kt0 * kTileKeys, item.ctx); u < b1; ++u) {
    if (!(seen_bits(mrow, P.mask_words, item.q_len, u - item.ctx) & 1)) continue;
    const int id = __ldg(P.bt + static_cast<int64_t>(item.seq) * P.max_blocks + u / kBlock);
    if (id < 0 || id >= P.num_blocks) continue;
    const __nv_bfloat16* src = P.v_cache + ((static_cast<int64_t>(id) * P.hkv + item.head) * kBlock + u % kBlock) * 128;
#pragma unroll 1
    for (int e = 0; e < 128; ++e) {
      const float x = __bfloat162float(src[e]);
      if (isfinite(x)) continue;
      if (item.slot >= 0) {
        reinterpret_cast<float*>(dst)[e] += x;
      } else {
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(dst) + e;
        *o = __float2bfloat16_rn(__bfloat162float(*o) + x);
      }
    }
  }
}

// (Code size: the streams, the MMA thread and the producers run different code by turns.  With every
// loop below unrolled, two thirds of the instruction fetches missed the SM's cache and all of its
// warps waited for instructions: 64 requests of 128..4096 keys took a third longer.)
template <int kRuns>
__device__ void softmax_warps(const Params& P, Ctl& c, uint8_t* vbuf, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3;        // TMEM lane quarter of this warp
  const int w = (warp - 2) >> 2;  // its stream
  const int k = kRuns == 2 ? w : 0;     // its item ring
  const int tile = kRuns == 2 ? 0 : w;  // its row tile of an item
  const int r = wq * 32 + lane;         // its row
  const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t srow = tmem + lane_off + 128u * w, orow = tmem + lane_off + kOCol + 128u * w;
  volatile int* abort_flag = &c.abort_flag;
  uint32_t tiles = 0;  // of this stream's run
  uint32_t it = 0, tc = 0, oc = 0, before = 0;
  bool ok = true;
  const int row = r - P.row0[w];  // the row within the item's row tile (below 0: none)
  const int rj = row >> P.gp_log2, rg = r & (P.gp - 1);
  const float scale = P.scale_log2;
  const float sign = scale >= 0.f ? 1.f : -1.f;

  while (ok) {
    const int slot = it % kRing;
    if (!wait_for(&c.item_full[k][slot], (it / kRing) & 1, abort_flag)) {
      ok = false;
      break;
    }
    const Item& item = c.ring[k][slot];  // stays until this warp gives the slot back
    ++it;
    if (item.idx < 0) break;
    const int nt = item.nt, nq = item.nq[tile];
    if (nq == 0) {  // the item has one row tile only
      tiles += nt;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.item_empty[k][slot]);
      continue;
    }
    const int ctx = item.ctx, q_len = item.q_len, kt0 = item.kt0;
    // this stream is the last one to read the item's tiles, and looks through their V rows
    const bool releases = kRuns == 2 || w == 1 || item.nq[1] == 0, cleans = kRuns == 2 || w == 0;
    const bool live = rj >= 0 && rj < nq && rg < P.group;  // a real (node, head) row
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint64_t* mrow = P.mask + (static_cast<int64_t>(item.t0) + item.j0[tile] + (live ? rj : 0)) * P.mask_words;
    float m_ref = -INFINITY, l_sum = 0.f;

    for (int j = 0; j < nt; ++j) {
      const int k0 = (kt0 + j) * kTileKeys;
      const bool drafted = k0 + kTileKeys > ctx;  // the tile holds keys that not every row sees
      const bool masked = drafted || sign < 0.f;  // (a negative scale wants the minimum)
      uint32_t vis[4];
      if (masked && warp_live) {
        const uint64_t lo = seen_bits(mrow, P.mask_words, q_len, k0 - ctx);
        const uint64_t hi = seen_bits(mrow, P.mask_words, q_len, k0 - ctx + 64);
        vis[0] = static_cast<uint32_t>(lo);
        vis[1] = static_cast<uint32_t>(lo >> 32);
        vis[2] = static_cast<uint32_t>(hi);
        vis[3] = static_cast<uint32_t>(hi >> 32);
      }
      if (!wait_for(&c.s_full[w], tc & 1, abort_flag)) {
        ok = false;
        break;
      }
      ++tc;
      tc_fence_after();
      // S of this tile is complete, and with it every MMA issued before: K has been read, and
      // V of the tile before
      const uint32_t n = c.number[k][tiles++ % 8];  // the tile's number in the rings
      if (r == 0 && releases) {
        mbar_arrive(&c.kempty[n % kKStages]);
        if (j > 0) mbar_arrive(&c.vempty[before % kVStages]);
      }
      before = n;
      // Before the first half of P is handed over, V of this key tile has landed and is clean.
      bool v_ok = true;
      auto first_half = [&]() {
        if (warp_live) tmem_st_wait();
        v_ok = wait_for(&c.vfull[n % kVStages], (n / kVStages) & 1, abort_flag);
        if (!v_ok) return;
        if (drafted && cleans && k0 + r >= ctx &&
            clean_v_row(vbuf + (n % kVStages) * kTileBytes, r, k0 + r >= ctx + q_len))
          *reinterpret_cast<volatile int*>(&c.spoilt[k][slot]) = 1;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.p_full[w][0]);
      };
      if (warp_live) {
        // (a row that sees nothing of the tile has no maximum)
        const float raw = masked ? row_extremum_bits(srow, vis, sign) : row_extremum<true, false>(srow, kTileKeys);
        const float tmax = raw == -INFINITY ? -INFINITY : raw * (scale * sign);
        if (j == 0) {
          m_ref = tmax;
        } else {
          const bool need = tmax > m_ref + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = need ? tmax : m_ref;
            const float alpha = need ? exp2f(m_ref - m_new) : 1.f;
#pragma unroll 1  // rare, and small in the instruction cache
            for (int ch = 0; ch < 8; ++ch) {
              uint32_t v[16];
              tmem_ld16_sync(orow + 16 * ch, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              tmem_st16(orow + 16 * ch, v);
            }
            tmem_st_wait();
            l_sum *= alpha;
            m_ref = m_new;
          }
        }
        // a row that has seen nothing yet: all its weights are 0
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        l_sum += masked ? row_exp_to_p_bits(srow, vis, scale, m_use, first_half)
                        : kRuns == 1 ? row_exp_to_p<false>(srow, kTileKeys, scale, m_use, first_half)
                                     : row_exp_to_p_loop(srow, scale, m_use, first_half);
        tmem_st_wait();
      } else {
        first_half();  // (no row of this warp is stored: its P may hold anything)
      }
      if (!v_ok) {
        ok = false;
        break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.p_full[w][1]);
    }
    if (!ok) break;
    if (!wait_for(&c.o_full[w], oc++ & 1, abort_flag)) {
      ok = false;
      break;
    }
    tc_fence_after();
    if (r == 0 && releases) mbar_arrive(&c.vempty[before % kVStages]);
    const bool bad = c.bad[k][slot] != 0;
    const int part = item.slot;
    // where the row goes: the output, or its partial
    uint8_t* dst;
    if (part < 0)
      dst = reinterpret_cast<uint8_t*>(P.out + ((static_cast<int64_t>(item.t0) + item.j0[tile] + rj) * P.hq +
                                                static_cast<int64_t>(item.head) * P.group + rg) * 128);
    else
      dst = reinterpret_cast<uint8_t*>(P.part_o + (static_cast<int64_t>(part) * P.rows_cap + 128 * tile + row) * 128);
    const bool zero = bad || l_sum == 0.f;
    const float inv = 1.f / l_sum;
#pragma unroll 1  // half of the row at a time keeps the code and the registers small
    for (int g = 0; g < 2; ++g) {
      uint32_t v[2][32];
      tmem_ld32_issue(orow + 64 * g, v[0]);
      tmem_ld32_issue(orow + 64 * g + 32, v[1]);
      tmem_ld32_wait(v[0]);
      tmem_ld32_wait(v[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (live && part >= 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st_global_v8(dst + 256 * g + 128 * h + 32 * q, *reinterpret_cast<const uint32_t(*)[8]>(v[h] + 8 * q));
        } else if (live) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t wv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(v[h][16 * q + 2 * e]) * inv,
                                                              __uint_as_float(v[h][16 * q + 2 * e + 1]) * inv);
              wv[e] = zero ? 0u : *reinterpret_cast<const uint32_t*>(&h2);
            }
            uint8_t* to = dst + 128 * g + 64 * h + 32 * q;
            if (P.out_v8) {
              st_global_v8(to, wv);
            } else {
              reinterpret_cast<uint4*>(to)[0] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
              reinterpret_cast<uint4*>(to)[1] = make_uint4(wv[4], wv[5], wv[6], wv[7]);
            }
          }
        }
        __syncwarp();
      }
    }
    if (live && part >= 0) {  // maximum and sum (a sum of -1: a bad block id)
      float* ml = P.part_ml + (static_cast<int64_t>(part) * P.rows_cap + 128 * tile + row) * 2;
      ml[0] = m_ref;
      ml[1] = bad ? -1.f : l_sum;
    }
    // O has been read: the next item's first P V may overwrite it
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.o_free[w]);
    if (live && !bad && *reinterpret_cast<volatile int*>(&c.spoilt[k][slot]) != 0)
      give_back(P, item, mrow, kt0, nt, dst);
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.item_empty[k][slot]);
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
}

// The kernel cannot run as it is laid out: the call reports a failure, and nothing is merged.
__device__ __noinline__ void refuse_to_run(const Params& P, int runs) {
  if (threadIdx.x == 0) flag_error(P.err, kErrTimeout);
  if (threadIdx.x < 2 * runs) P.cuts[2 * ((threadIdx.x >> 1) * gridDim.x + blockIdx.x) + (threadIdx.x & 1)].parts = 0;
}

template <bool kPairs>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ CUtensorMap qmap,
                                                           const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap, const Params P) {
  constexpr int kRuns = kPairs ? 1 : 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // the swizzled tiles need it, and no room is left to round up in
    grid_dep_wait();
    refuse_to_run(P, kRuns);
    return;
  }
  uint8_t* qbuf = smem_raw;
  uint8_t* kbuf = qbuf + 2 * kTileBytes;
  uint8_t* vbuf = kbuf + kKStages * kTileBytes;
  Ctl& c = *reinterpret_cast<Ctl*>(vbuf + kVStages * kTileBytes);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&c.kfull[s], 1);
      mbar_init(&c.kempty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&c.vfull[s], 1);
      mbar_init(&c.vempty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&c.s_full[w], 1);
      mbar_init(&c.p_full[w][0], 4);
      mbar_init(&c.p_full[w][1], 4);
      mbar_init(&c.o_full[w], 1);
      mbar_init(&c.o_free[w], 4);
      mbar_init(&c.q_full[w], 1);
      mbar_init(&c.q_free[w], 1);
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&c.item_full[w][s], 1);
        mbar_init(&c.item_empty[w][s], kPairs ? 10 : 6);  // MMA thread, V producer, softmax warps
      }
      c.run[w].seq = 0;
      c.run[w].base = 0;
    }
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    c.q_loads[0] = c.q_loads[1] = 0;
    fence_mbar_init();
    tma_prefetch_map(&qmap);
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  if (warp == 1) tmem_alloc(&c.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all of it, which begins at the first column: constants need no registers
  grid_dep_wait();
  grid_dep_launch();
  if (c.tmem_base != tmem) {
    refuse_to_run(P, kRuns);
    if (warp == 1) {
      tmem_dealloc(c.tmem_base, kTmemCols);
      tmem_relinquish();
    }
    return;
  }
  if (P.num_seqs > kFewSeqs) find_runs<kRuns>(P, c);
  else if (warp == 0) find_runs_few<kRuns>(P, c);
  if (warp == 0 || warp == 10)
    producer_warp<kRuns>(P, warp == 0, &qmap, warp == 0 ? &kmap : &vmap, c, qbuf, warp == 0 ? kbuf : vbuf);
  else if (warp == 1)
    mma_warp<kRuns>(P, c, qbuf, kbuf, vbuf, tmem);
  else
    softmax_warps<kRuns>(P, c, vbuf, tmem);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
    tmem_relinquish();
  }
}

// ------------------------------------------------------------------ merge
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const Params P) {
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  join_rows<4>(
      P.cuts, P.part_o, P.part_ml, P.rows_cap,
      [&](const Cut& cut, int row) {
        return ((row & 127) >> P.gp_log2) < (row >> 7 ? cut.rows[1] : cut.rows[0]) && (row & (P.gp - 1)) < P.group;
      },
      [&](const Cut& cut, int row, const Joined<4>& j) {
        const bool zero = j.bad || j.l == 0.f;
        const float inv = 1.f / j.l;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(j.o[0] * inv, j.o[1] * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(j.o[2] * inv, j.o[3] * inv);
        const uint2 packed = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        const int64_t t = static_cast<int64_t>(cut.t0) + (row >> 7 ? cut.first[1] : cut.first[0]) + ((row & 127) >> P.gp_log2);
        const int64_t at = (t * P.hq + static_cast<int64_t>(cut.head) * P.group + (row & (P.gp - 1))) * 128;
        reinterpret_cast<uint2*>(P.out + at)[lane] = zero ? make_uint2(0, 0) : packed;
      });
}

int gp_log2_of(int group) {
  int g = 0;
  while ((1 << g) < group) ++g;
  return g;
}

struct Layout {
  int rows_cap;
  size_t o_bytes, ml_bytes, bytes;
};
Layout layout_of(int32_t group, int32_t max_query_len, int num_sms, bool pairs) {
  Layout l;
  const int64_t rows = static_cast<int64_t>(max_query_len) << gp_log2_of(group), most = pairs ? 256 : 128;
  l.rows_cap = static_cast<int>(rows < most ? rows : most);
  const size_t runs = (pairs ? 1 : 2) * static_cast<size_t>(num_sms);
  const size_t slots = 2 * runs * l.rows_cap;
  l.o_bytes = slots * 128 * sizeof(float);
  l.ml_bytes = (slots * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255);
  l.bytes = l.o_bytes + l.ml_bytes + 2 * runs * sizeof(Cut);
  return l;
}

}  // namespace

size_t tree_tc_workspace(int32_t group, int32_t max_query_len, int num_sms) {
  return layout_of(group, max_query_len, num_sms, false).bytes;  // (the other is never larger)
}

int launch_tree_tc(const TreeArgs& t, void* workspace, int num_sms, uint32_t* err, cudaStream_t s) {
  const AttnArgs& a = t.a;
  const int hkv = a.cache.num_kv_heads, group = a.num_q_heads / hkv;
  const uint64_t rows = static_cast<uint64_t>(a.cache.num_blocks) * hkv * kBlock;
  if (rows >= (1ull << 31)) return PKV_ERR_UNSUPPORTED;
  Params p{};
  p.gp_log2 = gp_log2_of(group);
  p.gp = 1 << p.gp_log2;
  p.rows_q = kTileKeys / p.gp;
  CUtensorMap qm, km, vm;
  int st = encode_tensor_map_2d(&km, a.k_cache, 128, rows, 256, 64, 16);
  if (st) return st;
  st = encode_tensor_map_2d(&vm, a.v_cache, 128, rows, 256, 64, 16);
  if (st) return st;
  const uint64_t qdims[3] = {128, static_cast<uint64_t>(a.num_q_heads), static_cast<uint64_t>(a.num_tokens)};
  const uint64_t qstrides[2] = {256, static_cast<uint64_t>(a.num_q_heads) * 256};
  const uint32_t qbox[3] = {64, static_cast<uint32_t>(p.gp), static_cast<uint32_t>(p.rows_q)};
  st = encode_tensor_map_3d(&qm, a.q, qdims, qstrides, qbox);
  if (st) return st;
  // Requests with more rows than a tile share K and V between two of them, if they are long: 68 requests
  // with 12 / 4 heads and 61 nodes each take 68, 100 us with 1500, 3000 keys, and 92, 153 in single row
  // tiles.  For short ones a unit's beginning and end count more, which streams that work for
  // themselves have twice as fast: 6 such requests of 40, 200, 400 keys take 9.9, 14.8, 16.5 us (14.6,
  // 19.5, 18.1 in pairs), 68 of 400 with 2 to 61 nodes 32.5 (33.1).  Where no request has more rows than
  // a tile, the second stream of a pair would rest: one request of 7 nodes 9.7 us (12.3 in pairs), 64 of
  // 20..300 keys and 16 nodes 28.6 (31.5); what reads enough is bound by that (64 of 128..4096: 101.5 both).
  const bool pairs = a.max_query_len > p.rows_q && a.max_seq_len > kShortKeys;
  p.unit_q = pairs ? 2 * p.rows_q : p.rows_q;
  p.unit_q_log2 = 7 - p.gp_log2 + (pairs ? 1 : 0);
  // CTAs: one per SM, fewer where the caller's bounds leave less to do
  const int runs_per_cta = pairs ? 1 : 2;
  const int64_t units = (static_cast<int64_t>(a.max_query_len) + p.unit_q - 1) / p.unit_q * hkv;
  const int64_t key_tiles = (static_cast<int64_t>(a.max_seq_len) + kTileKeys - 1) / kTileKeys;
  const int64_t tiles = units >= 2 * num_sms ? units : units * key_tiles;  // (enough to know)
  const int64_t most = tiles >= 2 * num_sms ? 2 * num_sms : tiles * a.num_seqs;
  const int min_tiles = pairs ? 2 : 1;
  const int ctas = static_cast<int>(most < min_tiles * num_sms ? (most + min_tiles - 1) / min_tiles : num_sms);
  p.unit_cost = most < 2 * num_sms ? 0 : 2;
  p.min_run = min_tiles + p.unit_cost;
  const Layout l = layout_of(group, a.max_query_len, num_sms, pairs);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.bt = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.mask = t.mask;
  p.err = err;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.o_bytes);
  p.cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(workspace) + l.o_bytes + l.ml_bytes);
  p.num_blocks = a.cache.num_blocks;
  p.num_tokens = a.num_tokens;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.max_q = a.max_query_len;
  p.mask_words = t.mask_words;
  p.hkv = hkv;
  p.hq = a.num_q_heads;
  p.group = group;
  p.rows_cap = l.rows_cap;
  p.out_v8 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0 ? 1 : 0;
  // Few rows: a warp takes as long for one live row as for 32, so the streams' live rows go to
  // different SM sub-partitions (a warp's TMEM quarter is its sub-partition): 101.5 instead of 101.8
  // us for 64 requests of 16 nodes.
  if (!pairs && l.rows_cap <= 64) p.row0[1] = 64;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  auto* kernel = pairs ? tree_kernel<true> : tree_kernel<false>;
  static uint64_t smem_set[2] = {0, 0};
  st = set_smem_once(reinterpret_cast<const void*>(kernel), kSmemBytes, &smem_set[pairs ? 1 : 0]);
  if (st) return st;
  st = cuda_status(launch_k(kernel, dim3(ctas), dim3(kThreads), kSmemBytes, s, qm, km, vm, p));
  if (st) return st;
  return cuda_status(launch_k(tree_merge_kernel, dim3(2 * ctas * runs_per_cta, merge_ctas(l.rows_cap)), dim3(kMergeThreads), 0, s, p));
}

}  // namespace pkv
