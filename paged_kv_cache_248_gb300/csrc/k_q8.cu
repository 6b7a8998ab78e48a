// k_q8.cu -- attention over a paged cache in 8 bits (e4m3 codes, a scale for each block and kv head) on
// tcgen05 tensor cores.
//
// Mathematics.  With K_u = ks code_u and V_u = vs code_u, out = sum_u softmax_u(scale q.K_u) V_u over the keys
// that a query sees (causal, aligned to the context's end), in one pass with a running maximum and sum.
//
// The codes go from the cache to the tensor core as they are: they are the A operand of both products
// (S^T = K Q^T and O^T = V^T P^T, 128 keys, or 128 elements of V, by the rows of a unit), and nothing of a
// tile is converted or written a second time.  Turning a tile into bf16 on the way would move each byte through
// shared memory six times where two will do, which is more than it has bandwidth for at HBM's rate.
// The other operands, queries and weights, are split into e4m3 terms side by side in the columns:
//   q = (hi + lo / 32) / c, c a power of two for a unit's rows: a bf16 has 8 significant bits, two terms of 4
//     each give them exactly, down to 2^-22 of the unit's largest element;
//   p = hi + mid / 16 + lo / 512 of a weight p rounded to fp16 (2^-11): three terms hold it down to 2^-19,
//     2^-25 of a row's largest weight at least, so that a hundred thousand small weights beside a large
//     one keep their share, which two terms (2^-20) do not.
// Scales: ks multiplies a key's scores.  vs goes into the weight, as log2 vs added to the score, so that a row's
// reference is the largest w vs of it, and out again of the row's sum, which takes p / vs.
// Scores, maxima, sums and accumulators are fp32.
//
// Rows.  The G query heads of a kv head and consecutive tokens are folded into the rows of a unit, GP = G
// rounded up to a power of two: 16 rows (one warpgroup of softmax) where every request brings one
// token, else 64 (two warpgroups, 32 each, which share the K and V tiles).  A softmax thread is one key of the
// tile: masks are a threshold on the row number, scales are its own, and its row sums stay in registers until the
// unit ends.  The reference of a row moves only when a score of the tile exceeds it by 2^3, which a vote of
// the warpgroup tells; only then is a maximum taken across the threads and O rescaled.
//
// Cut.  All units' key tiles, one after the other (and some places more for each unit's beginning and end), are
// cut into equal runs, one a CTA, which derives its run from the lengths by itself; a unit that is cut
// leaves partial rows, joined by the merge kernel (tree_merge.cuh).
//
// Per CTA: warp 0 walks the run and loads K and V by TMA (16 rows of 128 bytes a block, 128-byte swizzle), warp 1
// issues the MMAs, the others are softmax.  All waits are bounded (ptx.cuh).
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "pkv_internal.cuh"
#include "tree_merge.cuh"

namespace pkv {
namespace {

constexpr int kHalfTile = kTileKeys * 128;  // K or V of a tile, bytes
constexpr int kRing = 4;                    // items published ahead
constexpr int kBlocksPerTile = kTileKeys / kBlock;
constexpr float kTop = 5.75f;         // log2 of a row's largest weight when its reference is set
constexpr float kMost = 8.75f;        // and the most that it may reach: 2^8.75 < 448
constexpr float kLeastV = 8.271806125530277e-25f, kMostV = 1.298074214633707e33f;  // 2^-80, 2^110

template <int kGroups>  // softmax warpgroups
struct Shape {
  static constexpr int kRows = kGroups == 1 ? 16 : 32;  // of a warpgroup
  static constexpr int kOctets = kRows / 8;
  static constexpr int kStages = kGroups == 1 ? 3 : 5;
  static constexpr int kThreads = 64 + 128 * kGroups;
  static constexpr int kCtasPerSm = kGroups == 1 ? 2 : 1;
  static constexpr int kQBytes = 2 * kRows * 128;
  static constexpr int kPBytes = (24 * kOctets + 15) / 16 * 2048;
  // tensor memory columns of a warpgroup: S of even and of odd tiles, O
  static constexpr uint32_t kSCols = 2 * kRows, kOCol = 2 * kSCols, kCols = kGroups == 1 ? 128 : 256;
  static constexpr uint32_t kTmem = kCols * kGroups;
};

// A part of a unit: what one run does of it.
struct alignas(16) Item {
  int32_t idx;  // -1: the run is over
  int32_t seq, head, slot;  // slot: where its partial goes, -1: the unit is finished here
  int32_t t0, ctx, len, j0;
  int32_t nq, kt0, nt, pad;
};

template <int kGroups>
struct Ctl {
  using S = Shape<kGroups>;
  uint64_t kfull[S::kStages], vfull[S::kStages], empty[S::kStages];
  uint64_t s_full[kGroups][2], p_full[kGroups], pv_done[kGroups], q_full[kGroups];
  uint64_t item_full[kRing], item_empty[kRing];
  uint64_t cleaned[2];  // V of an edge tile, by turns
  uint64_t drain;
  Item ring[kRing];
  int bad[kRing];
  float4 across[kGroups][S::kRows];  // a row's values of the four warps
  float largest[kGroups][4];
  uint8_t spoilt[2][kTileKeys];
  int64_t run_begin, run_end, run_base, run_len;
  int32_t run_seq;
  int64_t warp_sum[S::kThreads / 32];
  uint32_t tmem_base;
  int abort_flag;
};

template <int kGroups>
constexpr int smem_bytes() {
  using S = Shape<kGroups>;
  return S::kStages * 2 * kHalfTile + kGroups * (S::kQBytes + S::kPBytes) + static_cast<int>(sizeof(Ctl<kGroups>)) + 1024;
}
static_assert(smem_bytes<1>() <= 115712 && smem_bytes<2>() <= 232448, "shared memory of the 8-bit attention");

struct Params {
  const __nv_bfloat16* q;
  const float2* scales;
  const int32_t *bt, *seq_lens, *qsl;
  __nv_bfloat16* out;
  uint32_t* err;
  float* part_o;   // [2 * runs][rows_cap][128]
  float* part_ml;  // [2 * runs][rows_cap][2]
  Cut* cuts;       // [2 * runs]
  int64_t num_blocks, num_tokens;
  int32_t num_seqs, max_blocks, max_q, hkv, hq, group, gp_log2, unit_q_log2, unit_cost, rows_cap, min_run, once;
  float scale_log2;
};

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
  __device__ __forceinline__ int32_t tiles(const Params& P, int u) const {
    const int64_t end = static_cast<int64_t>(u + 1) << P.unit_q_log2;
    const int32_t seen = len - q_len + static_cast<int32_t>(end < q_len ? end : q_len);
    return (seen - 1) / kTileKeys + 1;
  }
  // Places of the units before unit u <= units - 1, all of which have 2^unit_q_log2 tokens: ceil((ctx + v Q) / 128) =
  // floor((a + v) / (128 / Q)) with a = floor((ctx + 127) / Q), v from 1 to u.
  __device__ __forceinline__ int64_t before(const Params& P, int u) const {
    const int k = 7 - P.unit_q_log2;
    const int64_t a = (static_cast<int64_t>(len - q_len) + 127) >> P.unit_q_log2;
    return floors(a + u + 1, k) - floors(a + 1, k) + static_cast<int64_t>(u) * P.unit_cost;
  }
};

__device__ __forceinline__ Request make_request(const Params& P, int32_t q0, int32_t q1, int32_t len) {
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
  r.units = fits ? ((r.q_len - 1) >> P.unit_q_log2) + 1 : 0;
  r.head_cost = fits ? r.before(P, r.units - 1) + r.tiles(P, r.units - 1) + P.unit_cost : 0;
  return r;
}

__device__ __forceinline__ Request load_request(const Params& P, int i) {
  return make_request(P, __ldg(P.qsl + i), __ldg(P.qsl + i + 1), __ldg(P.seq_lens + i));
}

__device__ __noinline__ void zero_wrong(const Params& P) {
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
template <int kGroups>
__device__ __forceinline__ void find_run(const Params& P, Ctl<kGroups>& c) {
  constexpr int kThreads = Shape<kGroups>::kThreads;
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
    c.run_begin = begin;
    c.run_end = end;
    c.run_len = len;
  }
  if (begin >= first && begin < first + mine) {
    int64_t at = first;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int64_t places = load_request(P, i).head_cost * P.hkv;
      if (begin < at + places) {
        c.run_seq = i;
        c.run_base = at;
        break;
      }
      at += places;
    }
  }
  if (any_wrong) zero_wrong(P);
  __syncthreads();
}

// Walks the items of a run; the whole warp holds it, lane l the lengths of request rb + l.
struct Walk {
  int64_t pos, end, base;
  int i, rb;
  int32_t q0, q1, len;
};

// The next item (idx -1: none is left).
__device__ __forceinline__ Item next_item(const Params& P, Walk& k, int64_t run_len) {
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

template <int kGroups>
__device__ __forceinline__ void raise_abort(Ctl<kGroups>& c, uint32_t* err) {
  *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
  flag_error(err, kErrTimeout);
}

// ------------------------------------------------------------------ producer
template <int kGroups>
__device__ void producer_warp(const Params& P, const CUtensorMap* kmap, const CUtensorMap* vmap, Ctl<kGroups>& c, uint8_t* tiles) {
  using S = Shape<kGroups>;
  const int lane = threadIdx.x & 31, b = lane & 7;
  volatile int* abort_flag = &c.abort_flag;
  Walk walk{c.run_begin, c.run_end, c.run_base, c.run_seq, -64, 0, 0, 0};
  if (lane < 2) P.cuts[2 * blockIdx.x + lane].parts = 0;
  __syncwarp();
  const bool is_v = lane >= 8;
  const CUtensorMap* map = is_v ? vmap : kmap;
  const uint64_t drop = l2_policy_evict_first();
  uint32_t n = 0, s = 0, phase = 1;
  bool ok = true;
  for (uint32_t it = 0; ok; ++it) {
    const Item item = next_item(P, walk, c.run_len);
    const int slot = it % kRing;
    ok = mbar_wait(&c.item_empty[slot], ((it / kRing) & 1) ^ 1, abort_flag);
    if (!ok) break;
    if (lane == 0) {
      c.ring[slot] = item;
      c.bad[slot] = 0;
      mbar_arrive(&c.item_full[slot]);
    }
    __syncwarp();
    if (item.idx < 0) break;
    const int32_t last = (item.len - 1) / kBlock;
    const int32_t* row = P.bt + static_cast<int64_t>(item.seq) * P.max_blocks;
    const auto id_of = [&](int32_t tile) {
      const int32_t at = tile * kBlocksPerTile + b;
      return at <= last ? __ldg(row + at) : 0;
    };
    int32_t id = id_of(item.kt0);
    for (int32_t tile = item.kt0; tile < item.kt0 + item.nt; ++tile) {
      int32_t cur = id;
      if (tile + 1 < item.kt0 + item.nt) id = id_of(tile + 1);
      const bool wrong = cur < 0 || cur >= P.num_blocks;
      if (wrong) cur = 0;
      if (__any_sync(0xffffffffu, wrong)) {
        if (wrong && lane < 8) flag_error(P.err, kErrBlockId);
        // (read after the unit's last tile, which is loaded after this)
        if (lane == 0) *reinterpret_cast<volatile int*>(&c.bad[slot]) = 1;
        __syncwarp();
      }
      const int nblk = min(kBlocksPerTile, last + 1 - tile * kBlocksPerTile);
      ok = mbar_wait(&c.empty[s], phase, abort_flag);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&c.kfull[s], nblk * 2048);
      if (lane == 8) mbar_arrive_expect_tx(&c.vfull[s], nblk * 2048);
      __syncwarp();
      if (lane < 16 && b < nblk) {
        uint8_t* d = tiles + s * 2 * kHalfTile + (is_v ? kHalfTile : 0) + b * 2048;
        const int32_t y = (cur * P.hkv + item.head) * kBlock;
        uint64_t* bar = is_v ? &c.vfull[s] : &c.kfull[s];
        if (P.once) tma_load_2d(d, map, bar, 0, y, drop);
        else tma_load_2d(d, map, bar, 0, y);
      }
      ++n;
      if (++s == S::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
  __syncwarp();
  if (*abort_flag) {  // copies already issued land before the CTA's shared memory goes away
#pragma unroll 1
    for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i) {
      mbar_wait(&c.kfull[i % S::kStages], (i / S::kStages) & 1, nullptr);
      mbar_wait(&c.vfull[i % S::kStages], (i / S::kStages) & 1, nullptr);
    }
  }
}

// ------------------------------------------------------------------ MMA warp
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 8-row groups of warpgroup w of an item.
template <int kGroups>
__device__ __forceinline__ int octets_of(const Params& P, int nq, int w) {
  const int rows = (nq << P.gp_log2) - w * Shape<kGroups>::kRows;
  return max(0, min(Shape<kGroups>::kOctets, (rows + 7) / 8));
}

// One elected thread issues every MMA; the whole warp walks through the tiles.  A turn is S of the next
// tile, then P V of this one: MMAs complete in order, and S of tile j + 1 goes over S of tile j - 1, whose weights
// have been handed over by then.
template <int kGroups>
__device__ void mma_warp(const Params& P, Ctl<kGroups>& c, uint32_t tiles, uint32_t qbuf, uint32_t pbuf, uint32_t tmem) {
  using S = Shape<kGroups>;
  volatile int* abort_flag = &c.abort_flag;
  uint32_t n = 0, tc[kGroups] = {}, q_phase = 0;
  bool ok = true, issued = false;
  for (uint32_t it = 0;; ++it) {
    const int slot = it % kRing;
    ok = mbar_wait(&c.item_full[slot], (it / kRing) & 1, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const int nt = __shfl_sync(0xffffffffu, c.ring[slot].nt, 0), nq = __shfl_sync(0xffffffffu, c.ring[slot].nq, 0);
    const bool over = __shfl_sync(0xffffffffu, c.ring[slot].idx, 0) < 0;
    __syncwarp();
    if (over) break;
    if (elected()) mbar_arrive(&c.item_empty[slot]);
    int oct[kGroups];
#pragma unroll
    for (int w = 0; w < kGroups; ++w) {
      oct[w] = octets_of<kGroups>(P, nq, w);
      if (oct[w] > 0) {
        ok = ok && mbar_wait(&c.q_full[w], q_phase >> w & 1, abort_flag);
        q_phase ^= 1u << w;
      }
    }
    for (int j = -1; j < nt; ++j) {
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (j + 1 < nt) {
        const uint32_t m = n + j + 1, s = m % S::kStages;
        ok = ok && mbar_wait(&c.kfull[s], (m / S::kStages) & 1, abort_flag);
        tc_fence_after();
        const uint64_t a = umma_smem_desc(tiles + s * 2 * kHalfTile, 16, 1024, kLayout128B);
#pragma unroll
        for (int w = 0; w < kGroups; ++w) {
          if (oct[w] == 0) continue;
          const uint64_t b = umma_smem_desc(qbuf + w * S::kQBytes, 16, 1024, kLayout128B);
          const uint32_t idesc = umma_idesc_e4m3(128, 16 * oct[w], false, false), buf = (tc[w] + j + 1) & 1;
          if (elected()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_f8_ss(tmem + w * S::kCols + buf * S::kSCols, umma_desc_advance(a, 32 * k), umma_desc_advance(b, 32 * k), idesc,
                         k > 0);
            umma_commit(&c.s_full[w][buf]);
          }
          issued = true;
        }
      }
      if (j < 0) continue;
      const uint32_t m = n + j, s = m % S::kStages;
      ok = ok && mbar_wait(&c.vfull[s], (m / S::kStages) & 1, abort_flag);
      const uint64_t a = umma_smem_desc(tiles + s * 2 * kHalfTile + kHalfTile, kHalfTile, 1024, kLayout128B);
#pragma unroll
      for (int w = 0; w < kGroups; ++w) {
        if (oct[w] == 0) continue;
        ok = ok && mbar_wait(&c.p_full[w], (tc[w] + j) & 1, abort_flag);
        tc_fence_after();
        const uint64_t b = umma_smem_desc(pbuf + w * S::kPBytes, 128, 2048, kLayoutNone);
        const uint32_t idesc = umma_idesc_e4m3(128, (24 * oct[w] + 15) / 16 * 16, true, true);
        if (elected()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f8_ss(tmem + w * S::kCols + S::kOCol, umma_desc_advance(a, 4096 * k), umma_desc_advance(b, 512 * k), idesc,
                       j > 0 || k > 0);
          umma_commit(&c.pv_done[w]);
        }
        issued = true;
      }
    }
    if (!ok) break;
    n += nt;
#pragma unroll
    for (int w = 0; w < kGroups; ++w)
      if (oct[w] > 0) tc[w] += nt;
  }
  if (!ok && !*abort_flag && (threadIdx.x & 31) == 0) raise_abort(c, P.err);
  __syncwarp();
  // every MMA, and the arrivals that its commits trigger, is over before TMEM is freed
  if (issued) {
    if (elected()) umma_commit(&c.drain);
    mbar_wait(&c.drain, 0, nullptr);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ uint32_t to_e4m3(__half2 x) {
  return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 from_e4m3(uint32_t x) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x), __NV_E4M3));
}

__device__ __forceinline__ bool vote(int bar, bool x) {  // any of a warpgroup's threads
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(bar)
      : "memory");
  return r != 0;
}

// One of eight values over the lanes of a warp: lane l gets value l & 7, joined over the warp.
template <typename F>
__device__ __forceinline__ float join8(const float (&x)[8], F&& f) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
  const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = __shfl_xor_sync(0xffffffffu, h4 ? x[i] : x[i + 4], 4);
    a[i] = f(h4 ? x[i + 4] : x[i], y);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float y = __shfl_xor_sync(0xffffffffu, h2 ? a[i] : a[i + 2], 2);
    b[i] = f(h2 ? a[i + 2] : a[i], y);
  }
  const float y = __shfl_xor_sync(0xffffffffu, h1 ? b[0] : b[1], 1);
  float r = f(h1 ? b[1] : b[0], y);
  r = f(r, __shfl_xor_sync(0xffffffffu, r, 8));
  return f(r, __shfl_xor_sync(0xffffffffu, r, 16));
}

// Takes NaN codes out of row r of a V tile (all of a row behind the context), so that a weight of 0 can stand
// for a key that a row does not see.  Returns whether there was one that a row may see.
__device__ __noinline__ bool clean_v_row(uint8_t* vtile, int r, bool past) {
  uint4* row = reinterpret_cast<uint4*>(vtile + r * 128);
  bool spoilt = past;
  if (!past) {
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const uint4 x = row[(ch + r) & 7];  // (starting at another chunk in each lane spreads them over the banks)
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) spoilt |= __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
    }
  }
  if (spoilt) {
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) row[(ch + r) & 7] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  return spoilt && !past;
}

template <int kGroups>
__device__ __forceinline__ void softmax_warps(const Params& P, Ctl<kGroups>& c, uint8_t* tiles, uint8_t* qbuf, uint8_t* pbuf,
                                              uint32_t tmem) {
  using S = Shape<kGroups>;
  constexpr int kRows = S::kRows, kOctets = S::kOctets;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3, w = kGroups == 1 ? 0 : (warp - 2) >> 2;
  const int t = wq * 32 + lane;  // this thread's key of a tile, element of O
  const int bar = 1 + w;
  const uint32_t base = tmem + (static_cast<uint32_t>(wq * 32) << 16) + w * S::kCols;
  volatile int* abort_flag = &c.abort_flag;
  uint8_t* q = qbuf + w * S::kQBytes;
  uint8_t* p = pbuf + w * S::kPBytes;
  uint32_t n = 0, tc = 0, edges = 0;
  float unscale = 0.f;  // of the scores of the unit whose Q is in place: scale log2(e) / c
  bool ok = true;

  // The unit's rows of this warpgroup as e4m3 terms in Q (row r: hi at 16 (r / 8) + r % 8, lo 8 rows further).
  const auto load_q = [&](const Item& item) {
    constexpr int kPerRow = 128 / kRows;  // threads of a row, kRows elements each
    const int r = t / kPerRow, part = t % kPerRow, row = w * kRows + r;
    const int j = row >> P.gp_log2, g = row & ((1 << P.gp_log2) - 1);
    uint4 raw[kRows / 8] = {};
    if (j < item.nq && g < P.group) {
      const uint4* src = reinterpret_cast<const uint4*>(
          P.q + ((static_cast<int64_t>(item.t0) + item.j0 + j) * P.hq + static_cast<int64_t>(item.head) * P.group + g) * 128 + part * kRows);
#pragma unroll
      for (int i = 0; i < kRows / 8; ++i) raw[i] = __ldg(src + i);
    }
    float x[kRows], most = 0.f;
#pragma unroll
    for (int i = 0; i < kRows / 8; ++i) {
      const uint32_t y[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = __uint_as_float(y[e] << 16);
        x[8 * i + 2 * e + 1] = __uint_as_float(y[e] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      if (!(fabsf(x[e]) <= 3.4e38f)) x[e] = __int_as_float(0x7fffffff);  // (an infinity makes its row NaN, as 0 inf would)
      most = fmaxf(most, fabsf(x[e]));                                   // (NaN is passed over)
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (lane == 0) c.largest[w][wq] = __uint_as_float(top);
    named_bar_sync(bar, 128);
    most = fmaxf(fmaxf(c.largest[w][0], c.largest[w][1]), fmaxf(c.largest[w][2], c.largest[w][3]));
    // most c in [128, 256): a term's rest is at most 8 units, 256 in those of the next
    const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -119), 127);
    const float up = __int_as_float((127 + 7 - e) << 23);
    unscale = P.scale_log2 * (e >= -100 ? __int_as_float((127 - 7 + e) << 23) : 0.f);
    const int n_hi = 16 * (r >> 3) + (r & 7);
#pragma unroll
    for (int k = 0; k < kRows / 16; ++k) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = lo[i] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 y = make_float2(x[16 * k + 4 * i + 2 * h] * up, x[16 * k + 4 * i + 2 * h + 1] * up);
          const uint32_t code = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
          const float2 back = __half22float2(from_e4m3(code));
          hi[i] |= code << (16 * h);
          lo[i] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2((y.x - back.x) * 32.f, (y.y - back.y) * 32.f),
                                                                  __NV_SATFINITE, __NV_E4M3))
                   << (16 * h);
        }
      }
      const int ch = part * (kRows / 16) + k;
      *reinterpret_cast<uint4*>(q + n_hi * 128 + ((ch ^ (n_hi & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(q + (n_hi + 8) * 128 + ((ch ^ (n_hi & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.q_full[w]);
  };

  uint32_t it = 0;
  ok = mbar_wait(&c.item_full[0], 0, abort_flag);
  ok = !vote(bar, !ok);  // (what follows has barriers: all of the warpgroup's threads go on, or none)
  if (ok && c.ring[0].idx >= 0 && octets_of<kGroups>(P, c.ring[0].nq, w) > 0) load_q(c.ring[0]);
  while (ok) {
    const Item item = c.ring[it % kRing];
    if (item.idx < 0) break;
    const int octets = octets_of<kGroups>(P, item.nq, w);
    const bool alone = kGroups == 1 || octets_of<kGroups>(P, item.nq, 1) == 0;  // this warpgroup has all of the rows
    const float factor = unscale;
    float m[kRows], l[kRows];
    if (octets > 0) {
      const int32_t last = (item.len - 1) / kBlock, tile_end = item.kt0 + item.nt;
      const int32_t* row = P.bt + static_cast<int64_t>(item.seq) * P.max_blocks;
      // this thread's block of a tile, and its scales, a tile and two ahead
      const auto id_of = [&](int32_t tile) {
        const int32_t at = min(tile * kBlocksPerTile + (t >> 4), last);
        return __ldg(row + at);
      };
      const auto scales_of = [&](int32_t id) {
        return __ldg(P.scales + static_cast<int64_t>(id < 0 || id >= P.num_blocks ? 0 : id) * P.hkv + item.head);
      };
      float2 sc = scales_of(id_of(item.kt0));
      int32_t id = item.nt > 1 ? id_of(item.kt0 + 1) : 0;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        m[r] = 0.f;
        l[r] = 0.f;
      }
#pragma unroll 1
      for (int j = 0; j < item.nt; ++j, ++tc, ++n) {
        const int32_t tile = item.kt0 + j, key = tile * kTileKeys + t;
        const float2 now = sc;
        if (tile + 1 < tile_end) sc = scales_of(id);
        if (tile + 2 < tile_end) id = id_of(tile + 2);
        const float vs = fminf(fmaxf(now.y, kLeastV), kMostV);
        const float ks = now.x * factor, lv = __log2f(vs), iv = 1.f / vs;
        // row r sees the key if its token, j0 + (r >> gp_log2), does not come before it
        const int32_t ahead = key - item.ctx - item.j0;
        const int32_t r_min = key >= item.len ? kRows : min(max(ahead, 0), 64) * (1 << P.gp_log2) - w * kRows;
        const bool edge = (tile + 1) * kTileKeys > item.ctx + item.j0 + 1;  // not every row sees all of the tile
        const uint32_t s = n % S::kStages, buf = tc & 1;
        ok = mbar_wait(&c.s_full[w][buf], (tc >> 1) & 1, abort_flag);
        tc_fence_after();
        bool spoilt = false;
        if (edge) {
          // The first warpgroup looks through V and tells the second.  (It is at most one such tile ahead when
          // it comes here, since S of the tile after next waits for the second one's weights.)
          if (kGroups == 1 || w == 0) {
            ok = ok && mbar_wait(&c.vfull[s], (n / S::kStages) & 1, abort_flag);
            if (ok) spoilt = clean_v_row(tiles + s * 2 * kHalfTile + kHalfTile, t, key >= item.len);
          }
          if (kGroups == 2 && !alone) {
            if (w == 0) {
              c.spoilt[edges & 1][t] = spoilt;
              __syncwarp();
              if (lane == 0) mbar_arrive(&c.cleaned[edges & 1]);
            } else {
              ok = ok && mbar_wait(&c.cleaned[edges & 1], (edges >> 1) & 1, abort_flag);
              spoilt = c.spoilt[edges & 1][t] != 0;
            }
            ++edges;
          }
        }
        float x[kRows];
        float most = -INFINITY;
#pragma unroll
        for (int g = 0; g < kOctets; ++g) {
          if (g < octets) {
            uint32_t v[16];
            tmem_ld16_sync(base + buf * S::kSCols + 16 * g, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float score = fmaf(__uint_as_float(v[8 + e]), 1.f / 32.f, __uint_as_float(v[e]));
              float u = fmaf(score, ks, lv);
              if (spoilt) u = __int_as_float(0x7fffffff);
              if (8 * g + e < r_min) u = -INFINITY;
              x[8 * g + e] = u - m[8 * g + e];
              most = fmaxf(most, x[8 * g + e]);
            }
          }
        }
        // the weights of the tile before have been read, and its V: their places are free
        if (j > 0) {
          ok = ok && mbar_wait(&c.pv_done[w], (tc - 1) & 1, abort_flag);
          if (t == 0 && ok) {
            uint64_t* e = &c.empty[(n - 1) % S::kStages];
            mbar_arrive(e);
            if (kGroups == 2 && alone) mbar_arrive(e);
          }
        }
        // A row that sees no key of the run's first tile sees none of the later ones: every row gets its reference
        // there, or needs none.
        if (vote(bar, most > kMost || j == 0 || !ok)) {
          if (vote(bar, !ok)) {  // (a wait that some thread gave up ends here for all of them)
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kOctets; ++g) {
            if (g < octets) {
              const float top = join8(*reinterpret_cast<const float(*)[8]>(x + 8 * g), [](float a, float b) { return fmaxf(a, b); });
              if (lane < 8) reinterpret_cast<float*>(&c.across[w][8 * g + lane])[wq] = top;
            }
          }
          named_bar_sync(bar, 128);
#pragma unroll
          for (int g = 0; g < kOctets; ++g) {
            if (g < octets) {
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 y = c.across[w][8 * g + e];
                const float top = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
                // how far the reference moves
                const float more = j > 0 ? fmaxf(top - kTop, 0.f) : top > -INFINITY ? top - kTop : 0.f;
                x[8 * g + e] -= more;
                m[8 * g + e] += more;
                f[e] = j > 0 ? ex2_approx(-more) : 1.f;  // (nothing has been summed up before the first tile)
                l[8 * g + e] *= f[e];
              }
              if (j > 0) {
#pragma unroll 1
                for (int k = 0; k < 3; ++k) {
                  uint32_t v[8];
                  tmem_ld8_sync(base + S::kOCol + 24 * g + 8 * k, v);
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f[e]);
                  tmem_st8(base + S::kOCol + 24 * g + 8 * k, v);
                }
                tmem_st_wait();
              }
            }
          }
          named_bar_sync(bar, 128);  // (c.across may be written again)
        }
#pragma unroll
        for (int g = 0; g < kOctets; ++g) {
          if (g < octets) {
            uint32_t b[3][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int k = 0; k < 3; ++k) b[k][h] = 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = 8 * g + 4 * h + 2 * e;
                const float p0 = ex2_approx(x[r]), p1 = ex2_approx(x[r + 1]);
                l[r] = fmaf(p0, iv, l[r]);
                l[r + 1] = fmaf(p1, iv, l[r + 1]);
                const __half2 y = __floats2half2_rn(p0, p1);
                const uint32_t hi = to_e4m3(y);
                const __half2 y1 = __hmul2(__hsub2(y, from_e4m3(hi)), __float2half2_rn(16.f));
                const uint32_t mid = to_e4m3(y1);
                const __half2 y2 = __hmul2(__hsub2(y1, from_e4m3(mid)), __float2half2_rn(32.f));
                b[0][h] |= hi << (16 * e);
                b[1][h] |= mid << (16 * e);
                b[2][h] |= to_e4m3(y2) << (16 * e);
              }
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const int o = 3 * g + k;
              *reinterpret_cast<uint2*>(p + (o >> 1) * 2048 + t * 16 + (o & 1) * 8) = make_uint2(b[k][0], b[k][1]);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.p_full[w]);
      }
      if (!ok) break;
    } else {
      n += item.nt;
    }
    // the next unit's rows, while the last products run
    const uint32_t next = it + 1;
    ok = mbar_wait(&c.item_full[next % kRing], (next / kRing) & 1, abort_flag);
    ok = !vote(bar, !ok);
    if (!ok) break;
    if (c.ring[next % kRing].idx >= 0 && octets_of<kGroups>(P, c.ring[next % kRing].nq, w) > 0) load_q(c.ring[next % kRing]);
    if (octets > 0) {
#pragma unroll
      for (int g = 0; g < kOctets; ++g) {
        if (g < octets) {
          const float sum = join8(*reinterpret_cast<const float(*)[8]>(l + 8 * g), [](float a, float b) { return a + b; });
          if (lane < 8) reinterpret_cast<float*>(&c.across[w][8 * g + lane])[wq] = sum;
        }
      }
      ok = mbar_wait(&c.pv_done[w], (tc - 1) & 1, abort_flag);
      ok = !vote(bar, !ok);
      if (!ok) break;
      tc_fence_after();
      if (t == 0) {
        uint64_t* e = &c.empty[(n - 1) % S::kStages];
        mbar_arrive(e);
        if (kGroups == 2 && alone) mbar_arrive(e);
      }
      const bool bad = *reinterpret_cast<volatile int*>(&c.bad[it % kRing]) != 0;
      const int part = item.slot;
#pragma unroll
      for (int g = 0; g < kOctets; ++g) {
        if (g < octets) {
          uint32_t v[3][8];
#pragma unroll
          for (int k = 0; k < 3; ++k) tmem_ld8_sync(base + S::kOCol + 24 * g + 8 * k, v[k]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = w * kRows + 8 * g + e, jr = r >> P.gp_log2, hr = r & ((1 << P.gp_log2) - 1);
            if (jr >= item.nq || hr >= P.group) continue;
            const float4 y = c.across[w][8 * g + e];
            const float sum = (y.x + y.y) + (y.z + y.w);
            const float o = fmaf(__uint_as_float(v[2][e]), 1.f / 512.f,
                                 fmaf(__uint_as_float(v[1][e]), 1.f / 16.f, __uint_as_float(v[0][e])));
            if (part >= 0) {
              const int64_t at = static_cast<int64_t>(part) * P.rows_cap + r;
              P.part_o[at * 128 + t] = o;
              if (t == 0) {
                // (of a row that saw nothing, or a NaN, the sum says it all)
                P.part_ml[2 * at] = sum != 0.f && sum == sum ? m[8 * g + e] : -INFINITY;
                P.part_ml[2 * at + 1] = bad ? -1.f : sum;
              }
            } else {
              const int64_t at = (static_cast<int64_t>(item.t0) + item.j0 + jr) * P.hq + static_cast<int64_t>(item.head) * P.group + hr;
              P.out[at * 128 + t] = __float2bfloat16_rn(bad || sum == 0.f ? 0.f : o / sum);
            }
          }
        }
      }
      tc_fence_before();
      named_bar_sync(bar, 128);  // O and the sums have been read
    }
    if (t == 0) mbar_arrive(&c.item_empty[it % kRing]);
    it = next;
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
}

template <int kGroups>
__global__ void __launch_bounds__(Shape<kGroups>::kThreads, Shape<kGroups>::kCtasPerSm)
    q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Params P) {
  using S = Shape<kGroups>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* qbuf = tiles + S::kStages * 2 * kHalfTile;
  uint8_t* pbuf = qbuf + kGroups * S::kQBytes;
  Ctl<kGroups>& c = *reinterpret_cast<Ctl<kGroups>*>(pbuf + kGroups * S::kPBytes);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&c.kfull[s], 1);
      mbar_init(&c.vfull[s], 1);
      mbar_init(&c.empty[s], kGroups);
    }
    for (int w = 0; w < kGroups; ++w) {
      mbar_init(&c.s_full[w][0], 1);
      mbar_init(&c.s_full[w][1], 1);
      mbar_init(&c.p_full[w], 4);
      mbar_init(&c.pv_done[w], 1);
      mbar_init(&c.q_full[w], 4);
    }
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&c.item_full[s], 1);
      mbar_init(&c.item_empty[s], 1 + kGroups);  // MMA warp, softmax warpgroups
    }
    mbar_init(&c.cleaned[0], 4);
    mbar_init(&c.cleaned[1], 4);
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    c.run_seq = 0;
    c.run_base = 0;
    fence_mbar_init();
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem_base, S::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  grid_dep_wait();
  grid_dep_launch();
  find_run<kGroups>(P, c);
  if (warp == 0) producer_warp<kGroups>(P, &kmap, &vmap, c, tiles);
  else if (warp == 1) mma_warp<kGroups>(P, c, smem_u32(tiles), smem_u32(qbuf), smem_u32(pbuf), tmem);
  else softmax_warps<kGroups>(P, c, tiles, qbuf, pbuf, tmem);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
}

__global__ void __launch_bounds__(kMergeThreads) q8_merge_kernel(const Params P) {
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  join_rows<4>(
      P.cuts, P.part_o, P.part_ml, P.rows_cap,
      [&](const Cut& cut, int row) {
        return (row >> P.gp_log2) < cut.rows[0] && (row & ((1 << P.gp_log2) - 1)) < P.group;
      },
      [&](const Cut& cut, int row, const Joined<4>& j) {
        const bool zero = j.bad || j.l == 0.f;
        const float inv = 1.f / j.l;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(j.o[0] * inv, j.o[1] * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(j.o[2] * inv, j.o[3] * inv);
        const uint2 packed = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        const int64_t t = static_cast<int64_t>(cut.t0) + cut.first[0] + (row >> P.gp_log2);
        const int64_t at = (t * P.hq + static_cast<int64_t>(cut.head) * P.group + (row & ((1 << P.gp_log2) - 1))) * 128;
        reinterpret_cast<uint2*>(P.out + at)[lane] = zero ? make_uint2(0, 0) : packed;
      });
}

int gp_log2_of(int group) {
  int g = 0;
  while ((1 << g) < group) ++g;
  return g;
}

struct Layout {
  int groups, rows_cap, runs;
  size_t o_bytes, ml_bytes, bytes;
};
Layout layout_of(int32_t group, int32_t max_query_len, int num_sms) {
  Layout l;
  l.groups = max_query_len == 1 ? 1 : 2;
  l.rows_cap = l.groups == 1 ? 16 : 64;
  const int64_t rows = static_cast<int64_t>(max_query_len) << gp_log2_of(group);
  if (rows < l.rows_cap) l.rows_cap = static_cast<int>(rows);
  l.runs = num_sms * (l.groups == 1 ? Shape<1>::kCtasPerSm : Shape<2>::kCtasPerSm);
  const size_t slots = 2 * static_cast<size_t>(l.runs) * l.rows_cap;
  l.o_bytes = slots * 128 * sizeof(float);
  l.ml_bytes = (slots * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255);
  l.bytes = l.o_bytes + l.ml_bytes + 2 * l.runs * sizeof(Cut);
  return l;
}

}  // namespace

size_t q8_workspace(const pkv_cache_desc& c, int32_t num_q_heads, int32_t max_query_len, int num_sms) {
  return layout_of(num_q_heads / c.num_kv_heads, max_query_len, num_sms).bytes;
}

int launch_q8(const AttnArgs& a, const float* scales, void* workspace, int num_sms, uint32_t* err, cudaStream_t s) {
  const int hkv = a.cache.num_kv_heads, group = a.num_q_heads / hkv;
  const uint64_t rows = static_cast<uint64_t>(a.cache.num_blocks) * hkv * kBlock;
  if (rows >= (1ull << 31)) return PKV_ERR_UNSUPPORTED;
  const Layout l = layout_of(group, a.max_query_len, num_sms);
  CUtensorMap km, vm;  // (rows of 128 bytes)
  int st = encode_tensor_map_2d(&km, a.k_cache, 64, rows, 128, 64, 16);
  if (st) return st;
  st = encode_tensor_map_2d(&vm, a.v_cache, 64, rows, 128, 64, 16);
  if (st) return st;
  Params p{};
  p.gp_log2 = gp_log2_of(group);
  p.unit_q_log2 = l.groups == 1 ? 0 : 6 - p.gp_log2;
  // CTAs: all that fit, fewer where the caller's bounds leave less to do
  const int64_t units = (((static_cast<int64_t>(a.max_query_len) - 1) >> p.unit_q_log2) + 1) * hkv;
  const int64_t key_tiles = (static_cast<int64_t>(a.max_seq_len) + kTileKeys - 1) / kTileKeys;
  const int64_t tiles = units >= l.runs ? units : units * key_tiles;  // (enough to know)
  const int64_t most = tiles >= l.runs ? tiles : tiles * a.num_seqs;
  const int ctas = static_cast<int>(most < l.runs ? most : l.runs);
  p.unit_cost = most < l.runs ? 0 : 2;
  p.min_run = 1 + p.unit_cost;
  p.once = a.max_query_len <= (1 << p.unit_q_log2);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.scales = reinterpret_cast<const float2*>(scales);
  p.bt = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.err = err;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.o_bytes);
  p.cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(workspace) + l.o_bytes + l.ml_bytes);
  p.num_blocks = a.cache.num_blocks;
  p.num_tokens = a.num_tokens;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.max_q = a.max_query_len;
  p.hkv = hkv;
  p.hq = a.num_q_heads;
  p.group = group;
  p.rows_cap = l.rows_cap;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  static uint64_t smem_set[2] = {0, 0};
  if (l.groups == 1) {
    st = set_smem_once(reinterpret_cast<const void*>(q8_kernel<1>), smem_bytes<1>(), &smem_set[0]);
    if (!st) st = cuda_status(launch_k(q8_kernel<1>, dim3(ctas), dim3(Shape<1>::kThreads), smem_bytes<1>(), s, km, vm, p));
  } else {
    st = set_smem_once(reinterpret_cast<const void*>(q8_kernel<2>), smem_bytes<2>(), &smem_set[1]);
    if (!st) st = cuda_status(launch_k(q8_kernel<2>, dim3(ctas), dim3(Shape<2>::kThreads), smem_bytes<2>(), s, km, vm, p));
  }
  if (st) return st;
  return cuda_status(launch_k(q8_merge_kernel, dim3(2 * ctas, merge_ctas(l.rows_cap)), dim3(kMergeThreads), 0, s, p));
}

}  // namespace pkv
