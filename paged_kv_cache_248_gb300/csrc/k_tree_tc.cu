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
// nodes x GP heads (GP = G rounded up to a power of two).  A unit is (request, kv head, up to
// two row tiles) and runs over all of the request's key tiles of 128 keys.
//
// Cut.  All units' key tiles, one after the other, are cut into as many equal runs as there
// are CTAs (at least kMinTiles long), so that one long request and a thousand short ones keep
// every SM equally busy; a CTA derives its run from the lengths by itself, without a planning
// launch.  A unit that lies within one run is finished there; of one that is cut, each run
// leaves its rows' unnormalised accumulator, maximum and sum, and the merge kernel joins them
// in order.  A CTA leaves at most two such partials.
//
// Streams.  Two S/P/O accumulator sets live in TMEM, each with a warpgroup of its own, so that one
// softmax runs while the tensor core works for the other.  With two row tiles a stream is a row
// tile, and both read every key tile; with one, the streams take the key tiles by turns and are
// joined at the end through TMEM, whose lanes both warpgroups can read.  A step n is one S
// tile: stream n % 2, key tile n / 2 (two row tiles) or n (one).
//
// Per CTA (320 threads): warp 0 loads (TMA boxes of the blocks' 16-token rows, 128-byte
// swizzle, 2 K and 3 V tiles in flight), one thread of warp 1 issues the MMAs, warps 2-5 and
// 6-9 are the streams' softmax.  The tiles that hold drafted keys (the last one or two of a
// request) take their visibility from the mask row's bits, the others see every key.  Their V
// rows are looked through for values that are not finite: a zero weight times those would
// reach rows that do not see them, so they are taken out of the tile and given back, in the
// epilogue, to the rows that do.
//
// Bound: the K/V bytes, read once per two row tiles, up to about 256 rows a unit, where the
// tensor core and the exponents take as long.  All waits are bounded (ptx.cuh).
#include "ptx.cuh"
#include "pkv_internal.cuh"
#include "softmax_row.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 320;
constexpr int kKStages = 2;
constexpr int kVStages = 3;
constexpr int kHalfBytes = 16384;
constexpr int kTileBytes = 2 * kHalfBytes;  // 128 x 128 bf16 in two 64-column halves
constexpr int kRing = 4;
constexpr uint32_t kTmemCols = 512;  // S_0, S_1 (P over their first 64 columns), O_0, O_1
constexpr uint32_t kOCol = 256;
constexpr int kBlocksPerTile = kTileKeys / kBlock;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: O is rescaled when a row's maximum grows by > 2^8
constexpr int kMinTiles = 2;               // a run's least length: one key tile per stream

struct alignas(16) Item {
  int32_t idx;  // -1: the run is over
  int32_t seq, head, valid;
  int32_t t0, q_len, ctx, len;
  int32_t kt0, nt;        // key tiles kt0 .. kt0 + nt - 1
  int32_t two;            // two row tiles (else the streams share one)
  int32_t slot;           // partial slot, -1: the unit is finished here
  int32_t j0[2], nq[2];   // row tile w: its first node and how many
};

struct Ctl {
  uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages];
  uint64_t s_full[2], o_full[2], o_free[2], p_full[2][2], q_full[2], q_free[2];
  uint64_t item_full[kRing], item_empty[kRing];
  uint64_t joined, drain;
  Item ring[kRing];
  int bad[kRing];     // a block id outside of the pool
  int spoilt[kRing];  // a drafted V row that is not finite
  float ml[2][128][2];  // [stream][row]: maximum and sum
  int64_t run_begin, run_end, run_len, start_base;
  int64_t warp_sum[kThreads / 32];
  int32_t start_seq;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr int kSmemBytes = (2 + kKStages + kVStages) * kTileBytes + static_cast<int>(sizeof(Ctl));
static_assert(kSmemBytes <= 232448, "tree attention shared memory");

// What the merge kernel needs of a unit that a CTA begins and does not finish.
struct alignas(16) Cut {
  int32_t parts;  // runs that hold a part of it, 0: none
  int32_t head, t0, two;
  int32_t j0[2], nq[2];
};

struct Params {
  __nv_bfloat16* out;
  const __nv_bfloat16* v_cache;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* qsl;
  const uint64_t* mask;
  uint32_t* err;
  float* part_o;   // [2 * CTAs][rows_cap][128]
  float* part_ml;  // [2 * CTAs][rows_cap][2]
  Cut* cuts;       // [CTAs]
  int64_t num_blocks, num_tokens;
  int32_t num_seqs, max_blocks, max_q, mask_words;
  int32_t hkv, hq, group, gp, gp_log2, rows_q, rows_cap, out_v8;
  float scale_log2;
};

__device__ __forceinline__ void raise_abort(Ctl& c, uint32_t* err) {
  *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
  flag_error(err, kErrTimeout);
}

// ------------------------------------------------------------------ units
struct Request {
  int32_t t0, q_len, len, valid;
  int32_t tiles, units;  // key tiles of a unit; units of one kv head
  int64_t cost;          // key tiles of all its units (an invalid one: a unit that zeroes its rows)
};

__device__ __forceinline__ Request make_request(const Params& P, int32_t q0, int32_t q1, int32_t len) {
  Request r;
  const int64_t n = static_cast<int64_t>(q1) - q0;
  const bool rows = n > 0 && q0 >= 0 && q1 <= P.num_tokens;
  r.t0 = q0;
  r.q_len = rows ? static_cast<int32_t>(n) : 0;
  r.len = len;
  r.valid = rows && len >= n && n <= P.max_q && (static_cast<int64_t>(len) + kBlock - 1) / kBlock <= P.max_blocks;
  r.tiles = r.valid ? (len - 1) / kTileKeys + 1 : 1;
  r.units = r.valid ? (r.q_len + 2 * P.rows_q - 1) / (2 * P.rows_q) : 1;
  r.cost = rows ? (r.valid ? static_cast<int64_t>(P.hkv) * r.units * r.tiles : 1) : 0;
  return r;
}

__device__ __forceinline__ Request load_request(const Params& P, int i) {
  return make_request(P, __ldg(P.qsl + i), __ldg(P.qsl + i + 1), __ldg(P.seq_lens + i));
}

// This CTA's run of key tiles and the request it begins in (all threads).
__device__ void find_run(const Params& P, Ctl& c) {
  const int per = (P.num_seqs + kThreads - 1) / kThreads;
  const int i0 = min(static_cast<int>(threadIdx.x) * per, P.num_seqs), i1 = min(i0 + per, P.num_seqs);
  int64_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += load_request(P, i).cost;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) c.warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += c.warp_sum[w];
    total += c.warp_sum[w];
  }
  const int64_t even = (total + gridDim.x - 1) / gridDim.x;
  const int64_t run = even > kMinTiles ? even : kMinTiles;
  const int64_t begin = run * blockIdx.x, end = begin + run < total ? begin + run : total;
  if (threadIdx.x == 0) {
    c.run_begin = begin;
    c.run_end = end;
    c.run_len = run;
  }
  if (begin >= before && begin < before + mine) {
    for (int i = i0; i < i1; ++i) {
      const int64_t cost = load_request(P, i).cost;
      if (begin < before + cost) {
        c.start_seq = i;
        c.start_base = before;
        break;
      }
      before += cost;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------------ producer warp
__device__ void producer_warp(const Params& P, const CUtensorMap* qmap, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              Ctl& c, uint8_t* qbuf, uint8_t* kbuf, uint8_t* vbuf) {
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &c.abort_flag;
  int64_t pos = c.run_begin, base = c.start_base;
  const int64_t end = c.run_end, run = c.run_len;
  int i = c.start_seq, rb = 0;
  uint32_t it = 0, tk = 0;
  uint32_t qc[2] = {0, 0};
  bool ok = true, loaded = false;
  int32_t my_q0 = 0, my_q1 = 0, my_len = 0;  // lane l: request rb + l
  Cut cut{};
  while (ok) {
    Item info{};
    info.idx = -1;
    if (pos < end) {
      if (!loaded || i - rb >= 32) {
        rb = i;
        loaded = true;
        const int r = min(rb + lane, P.num_seqs - 1);
        my_q0 = __ldg(P.qsl + r);
        my_q1 = __ldg(P.qsl + r + 1);
        my_len = __ldg(P.seq_lens + r);
      }
      const int src = i - rb;
      const Request rq = make_request(P, __shfl_sync(0xffffffffu, my_q0, src), __shfl_sync(0xffffffffu, my_q1, src),
                                      __shfl_sync(0xffffffffu, my_len, src));
      if (pos >= base + rq.cost) {  // (cost 0 among them)
        base += rq.cost;
        if (++i >= P.num_seqs) pos = end;  // (lengths that changed meanwhile)
        continue;
      }
      const int64_t off = pos - base;
      const int64_t unit = off / rq.tiles;
      const int first = static_cast<int>(off - unit * rq.tiles);
      const int64_t room = end - pos;
      info.idx = 0;
      info.seq = i;
      info.valid = rq.valid;
      info.t0 = rq.t0;
      info.q_len = rq.q_len;
      info.len = rq.len;
      info.ctx = rq.len - rq.q_len;
      info.kt0 = first;
      info.nt = static_cast<int>(rq.tiles - first < room ? rq.tiles - first : room);
      const int p = static_cast<int>(unit % rq.units);
      info.head = static_cast<int>(unit / rq.units);
      for (int w = 0; w < 2; ++w) {
        info.j0[w] = (2 * p + w) * P.rows_q;
        info.nq[w] = max(0, min(P.rows_q, rq.q_len - info.j0[w]));
      }
      info.two = info.nq[1] > 0 ? 1 : 0;
      info.slot = -1;
      if (rq.valid && info.nt < rq.tiles) {
        info.slot = 2 * blockIdx.x + (first == 0 ? 1 : 0);
        if (first == 0) {
          const int64_t last = (base + (unit + 1) * rq.tiles - 1) / run;
          cut.parts = static_cast<int32_t>(last - blockIdx.x) + 1;
          cut.head = info.head;
          cut.t0 = info.t0;
          cut.two = info.two;
          for (int w = 0; w < 2; ++w) {
            cut.j0[w] = info.j0[w];
            cut.nq[w] = info.nq[w];
          }
        }
      }
      pos += info.nt;
    }
    const int slot = it % kRing;
    if (!mbar_wait(&c.item_empty[slot], ((it / kRing) & 1) ^ 1, abort_flag)) {
      ok = false;
      break;
    }
    if (lane == 0) {
      c.ring[slot] = info;
      c.bad[slot] = 0;
      c.spoilt[slot] = 0;
      mbar_arrive(&c.item_full[slot]);
    }
    __syncwarp();
    ++it;
    if (info.idx < 0) break;
    if (!info.valid) continue;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (w == 1 && !info.two) break;
      if (!mbar_wait(&c.q_free[w], (qc[w] & 1) ^ 1, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        uint8_t* q = qbuf + w * kTileBytes;
        mbar_arrive_expect_tx(&c.q_full[w], kTileBytes);
        const int32_t y = info.head * P.group, z = info.t0 + info.j0[w];
        tma_load_3d(q, qmap, &c.q_full[w], 0, y, z, l2_policy_evict_first());
        tma_load_3d(q + kHalfBytes, qmap, &c.q_full[w], 64, y, z, l2_policy_evict_first());
      }
      __syncwarp();
      ++qc[w];
    }
    if (!ok) break;
    const int32_t* btrow = P.bt + static_cast<int64_t>(info.seq) * P.max_blocks;
    const int blocks = (info.len - 1) / kBlock + 1;
    int at = info.kt0 * kBlocksPerTile + lane;  // this lane's block of the next key tile
    int id = lane < kBlocksPerTile && at < blocks ? __ldg(btrow + at) : 0;
    for (int j = 0; j < info.nt; ++j) {
      const int nblk = min(kBlocksPerTile, blocks - (info.kt0 + j) * kBlocksPerTile);
      int cur = id;
      at += kBlocksPerTile;  // the next tile's ids load while this one waits for its slots
      if (j + 1 < info.nt) id = lane < kBlocksPerTile && at < blocks ? __ldg(btrow + at) : 0;
      const bool wrong = lane < nblk && (cur < 0 || cur >= P.num_blocks);
      if (__any_sync(0xffffffffu, wrong)) {
        if (wrong) flag_error(P.err, kErrBlockId);
        if (wrong) cur = 0;
        if (lane == 0) c.bad[slot] = 1;
        __syncwarp();
      }
      const int32_t row = (cur * P.hkv + info.head) * kBlock;
      const int sk = tk % kKStages, sv = tk % kVStages;
      if (!mbar_wait(&c.kempty[sk], ((tk / kKStages) & 1) ^ 1, abort_flag)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&c.kfull[sk], static_cast<uint32_t>(nblk) * 4096u);
      __syncwarp();
      if (lane < nblk) {
        uint8_t* d = kbuf + sk * kTileBytes + lane * 2048;
        tma_load_2d(d, kmap, &c.kfull[sk], 0, row);
        tma_load_2d(d + kHalfBytes, kmap, &c.kfull[sk], 64, row);
      }
      // (an abort between the two leaves a K tile in flight without its V: counted below)
      const bool v_ok = mbar_wait(&c.vempty[sv], ((tk / kVStages) & 1) ^ 1, abort_flag);
      if (!v_ok) {
        mbar_wait(&c.kfull[sk], (tk / kKStages) & 1, nullptr);
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&c.vfull[sv], static_cast<uint32_t>(nblk) * 4096u);
      __syncwarp();
      if (lane < nblk) {
        uint8_t* d = vbuf + sv * kTileBytes + lane * 2048;
        tma_load_2d(d, vmap, &c.vfull[sv], 0, row);
        tma_load_2d(d + kHalfBytes, vmap, &c.vfull[sv], 64, row);
      }
      ++tk;
    }
  }
  if (lane == 0) P.cuts[blockIdx.x] = cut;
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
  if (*abort_flag) {
    // copies already issued land before the CTA's shared memory goes away
    for (uint32_t n = tk > static_cast<uint32_t>(kKStages) ? tk - kKStages : 0; n < tk; ++n)
      mbar_wait(&c.kfull[n % kKStages], (n / kKStages) & 1, nullptr);
    for (uint32_t n = tk > static_cast<uint32_t>(kVStages) ? tk - kVStages : 0; n < tk; ++n)
      mbar_wait(&c.vfull[n % kVStages], (n / kVStages) & 1, nullptr);
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (qc[w] > 0) mbar_wait(&c.q_full[w], (qc[w] - 1) & 1, nullptr);
  }
}

// ------------------------------------------------------------------ MMA warp
__device__ void mma_warp(const Params& P, Ctl& c, uint8_t* qbuf, uint8_t* kbuf, uint8_t* vbuf, uint32_t tmem) {
  if ((threadIdx.x & 31) == 0) {
    const uint32_t idesc_s = umma_idesc_bf16(128, 128, false, false);
    const uint32_t idesc_o = umma_idesc_bf16(128, 128, false, true);
    const uint64_t qdesc[2] = {umma_smem_desc(smem_u32(qbuf), 16, 1024, kLayout128B),
                               umma_smem_desc(smem_u32(qbuf + kTileBytes), 16, 1024, kLayout128B)};
    volatile int* abort_flag = &c.abort_flag;
    uint32_t it = 0, tiles = 0;
    uint32_t qc[2] = {0, 0}, pc[2] = {0, 0}, ic[2] = {0, 0};
    bool issued = false, ok = true;
    auto issue_pv = [&](int w, int sv, bool acc, int hf) {
      const uint64_t bd = umma_smem_desc(smem_u32(vbuf + sv * kTileBytes), kHalfBytes, 1024, kLayout128B);
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {
        const int kk = 4 * hf + k4;
        umma_f16_ts(tmem + kOCol + 128 * w, tmem + 128 * w + 8 * kk, umma_desc_advance(bd, kk * 2048), idesc_o,
                    (acc || kk > 0) ? 1u : 0u);
      }
    };
    auto issue_s = [&](int w, int q, int sk) {
      const uint64_t b = umma_smem_desc(smem_u32(kbuf + sk * kTileBytes), 16, 1024, kLayout128B);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
        umma_f16_ss(tmem + 128 * w, umma_desc_advance(qdesc[q], off), umma_desc_advance(b, off), idesc_s, kk > 0);
      }
    };
    while (ok) {
      const int slot = it % kRing;
      if (!mbar_wait(&c.item_full[slot], (it / kRing) & 1, abort_flag)) {
        ok = false;
        break;
      }
      const Item info = c.ring[slot];
      ++it;
      if (info.idx < 0) break;
      if (info.valid) {
        const int two = info.two, steps = two ? 2 * info.nt : info.nt;
        ok = mbar_wait(&c.q_full[0], qc[0] & 1, abort_flag) && (!two || mbar_wait(&c.q_full[1], qc[1] & 1, abort_flag));
        // Step n: P V of step n - 2 (the stream's last one), then S of step n.  MMAs of one
        // thread complete in order, so S of step n cannot overwrite the P that step n - 2's
        // P V reads, and its completion tells the softmax that O holds every tile before.
        for (int n = 0; n < steps + 2 && ok; ++n) {
          const int w = n & 1;
          if (n >= 2) {
            const int m = n - 2;
            const int sv = (tiles + (two ? m >> 1 : m)) % kVStages;
            if (!mbar_wait(&c.p_full[w][0], pc[w] & 1, abort_flag) ||
                (m < 2 && !mbar_wait(&c.o_free[w], (ic[w] & 1) ^ 1, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_pv(w, sv, m >= 2, 0);
            if (!mbar_wait(&c.p_full[w][1], pc[w] & 1, abort_flag)) {
              ok = false;
              break;
            }
            ++pc[w];
            tc_fence_after();
            issue_pv(w, sv, m >= 2, 1);
            if (n >= steps) umma_commit(&c.o_full[w]);
          }
          if (n < steps) {
            const int kt = two ? n >> 1 : n;
            const uint32_t tk = tiles + kt;
            if ((!two || w == 0) && !mbar_wait(&c.kfull[tk % kKStages], (tk / kKStages) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_s(w, two ? w : 0, tk % kKStages);
            umma_commit(&c.s_full[w]);
            if (kt == info.nt - 1) umma_commit(&c.q_free[two ? w : 0]);
            issued = true;
          }
          if (n == 0 && steps == 1) ++n;  // a single step has no second stream
        }
        tiles += info.nt;
        ++qc[0];
        ++ic[0];
        if (two) ++qc[1];
        if (steps > 1) ++ic[1];
      }
      if (!ok) break;
      mbar_arrive(&c.item_empty[slot]);
    }
    if (!ok && !*abort_flag) raise_abort(c, P.err);
    if (issued) {
      // every MMA, and the arrivals that its commits trigger, is over before TMEM is freed
      umma_commit(&c.drain);
      mbar_wait(&c.drain, 0, nullptr);
    }
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax warps
// Bits s .. s + 63 of what a row sees, counted from its first drafted key (s < 0: context,
// seen whole), without those past the draft.
__device__ __forceinline__ uint64_t seen_bits(const uint64_t* row, int words, int q_len, int s) {
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

// Whether some bf16 of the pair is an infinity or NaN.
__device__ __forceinline__ bool not_finite2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

// The pair with a zero in the place of each infinity or NaN.
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}

__device__ void softmax_warps(const Params& P, Ctl& c, uint8_t* vbuf, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3;        // TMEM lane quarter of this warp
  const int w = (warp - 2) >> 2;  // its stream
  const int r = wq * 32 + lane;   // its row
  const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t srow = tmem + lane_off + 128u * w, orow_t = tmem + lane_off + kOCol + 128u * w;
  volatile int* abort_flag = &c.abort_flag;
  uint32_t it = 0, tc = 0, tiles = 0, turns = 0;
  uint32_t ic[2] = {0, 0};
  bool ok = true;
  const int rj = r >> P.gp_log2, rg = r & (P.gp - 1);
  const float scale = P.scale_log2;
  const bool pos_scale = scale >= 0.f;

  while (ok) {
    const int slot = it % kRing;
    if (!mbar_wait(&c.item_full[slot], (it / kRing) & 1, abort_flag)) {
      ok = false;
      break;
    }
    const Item info = c.ring[slot];
    ++it;
    if (info.idx < 0) break;
    if (!info.valid) {  // a request whose lengths do not fit: its rows are zero
      if (r == 0 && w == 0) flag_error(P.err, kErrLength);
      const int64_t vecs = static_cast<int64_t>(info.q_len) * P.hq * 16;
      uint4* dst = reinterpret_cast<uint4*>(P.out) + static_cast<int64_t>(info.t0) * P.hq * 16;
      for (int64_t v = threadIdx.x - 64; v < vecs; v += 256) dst[v] = make_uint4(0, 0, 0, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.item_empty[slot]);
      continue;
    }
    const int two = info.two, steps = two ? 2 * info.nt : info.nt;
    const int tile = two ? w : 0;
    const int nq = tile ? info.nq[1] : info.nq[0], j0 = tile ? info.j0[1] : info.j0[0];
    const bool live = rj < nq && rg < P.group;      // a real (node, head) row
    const bool warp_live = __any_sync(0xffffffffu, live);
    const uint64_t* mrow = P.mask + (static_cast<int64_t>(info.t0) + j0 + (rj < nq ? rj : 0)) * P.mask_words;
    float m_ref = -INFINITY, l_sum = 0.f;

    for (int n = w; n < steps && ok; n += 2) {
      const int kt = two ? n >> 1 : n;
      const uint32_t vt = tiles + kt;
      const int sv = vt % kVStages;
      const int k0 = (info.kt0 + kt) * kTileKeys;
      const bool drafted = k0 + kTileKeys > info.ctx;  // the tile holds keys that not every row sees
      uint32_t vis[4];
      if (drafted && warp_live) {
        const uint64_t lo = seen_bits(mrow, P.mask_words, info.q_len, k0 - info.ctx);
        const uint64_t hi = seen_bits(mrow, P.mask_words, info.q_len, k0 - info.ctx + 64);
        vis[0] = static_cast<uint32_t>(lo);
        vis[1] = static_cast<uint32_t>(lo >> 32);
        vis[2] = static_cast<uint32_t>(hi);
        vis[3] = static_cast<uint32_t>(hi >> 32);
      }
      if (!mbar_wait(&c.s_full[w], tc & 1, abort_flag)) {
        ok = false;
        break;
      }
      ++tc;
      tc_fence_after();
      // S of this step is complete, and with it every MMA issued before: the K tile has been
      // read by its last reader, and so has the V tile of this stream's previous step
      if (r == 0 && (!two || w == 1)) {
        mbar_arrive(&c.kempty[vt % kKStages]);
        if (n >= 2) mbar_arrive(&c.vempty[(tiles + (two ? kt - 1 : kt - 2)) % kVStages]);
      }
      bool v_ok = true;
      // Before the first half of P is handed over, V of this key tile has landed, its rows
      // past the context are zero, and drafted rows that are not finite are taken out.
      auto first_half = [&]() {
        if (warp_live) tmem_st_wait();
        v_ok = mbar_wait(&c.vfull[sv], (vt / kVStages) & 1, abort_flag);
        if (!v_ok) return;
        if (drafted && (!two || w == 0) && k0 + r >= info.ctx) {
          // starting each lane at chunk r mod 8 spreads eight lanes over all banks
          uint8_t* vrow = vbuf + sv * kTileBytes + r * 128;
          const bool past = k0 + r >= info.len;
          bool wrote = past;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            const int off = ((ch + r) & 7) * 16;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint4* at = reinterpret_cast<uint4*>(vrow + half * kHalfBytes + off);
              if (past) {
                *at = make_uint4(0, 0, 0, 0);
                continue;
              }
              const uint4 x = *at;
              if (not_finite2(x.x) | not_finite2(x.y) | not_finite2(x.z) | not_finite2(x.w)) {
                *at = make_uint4(finite2(x.x), finite2(x.y), finite2(x.z), finite2(x.w));
                *reinterpret_cast<volatile int*>(&c.spoilt[slot]) = 1;
                wrote = true;
              }
            }
          }
          if (wrote) {
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.p_full[w][0]);
      };
      if (warp_live) {
        const float hidden = pos_scale ? -INFINITY : INFINITY;
        float raw;
        if (drafted) raw = pos_scale ? row_extremum_bits<true>(srow, vis) : row_extremum_bits<false>(srow, vis);
        else raw = pos_scale ? row_extremum<true, false>(srow, kTileKeys) : row_extremum<false, true>(srow, kTileKeys);
        const float tmax = raw == hidden ? -INFINITY : raw * scale;
        if (n < 2) {
          m_ref = tmax;
        } else {
          const bool need = tmax > m_ref + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = need ? tmax : m_ref;
            const float alpha = need ? exp2f(m_ref - m_new) : 1.f;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              uint32_t v[16];
              tmem_ld16_sync(orow_t + 16 * ch, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_st16(orow_t + 16 * ch, v);
            }
            tmem_st_wait();
            l_sum *= alpha;
            m_ref = m_new;
          }
        }
        // a row that has seen nothing yet: all its weights are 0
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
        l_sum += drafted ? row_exp_to_p_bits(srow, vis, scale, m_use, first_half)
                         : row_exp_to_p<false>(srow, kTileKeys, scale, m_use, first_half);
        if (v_ok) tmem_st_wait();
      } else {
        first_half();
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
    const uint32_t last_v = two ? info.nt - 1 : (info.nt - 1 - ((info.nt - 1 - w) & 1));  // this stream's last key tile
    const bool both = steps > 1;
    float a0 = 1.f, a1 = 0.f;  // weights of O_0 and O_1 (one row tile), of O_w (two)
    if (two) {
      if (!mbar_wait(&c.o_full[w], ic[w] & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (r == 0 && w == 1) mbar_arrive(&c.vempty[(tiles + last_v) % kVStages]);
    } else {
      // Both streams' maxima and sums, then their accumulators.  A stream's O being complete
      // (the first stream's, for one without a step) means that all eight warps have read
      // the unit before, so that ml may be written.
      const int mine = w < steps ? w : 0;
      if (!mbar_wait(&c.o_full[mine], ic[mine] & 1, abort_flag)) {
        ok = false;
        break;
      }
      c.ml[w][r][0] = m_ref;
      c.ml[w][r][1] = l_sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.joined);
      if (!mbar_wait(&c.joined, turns & 1, abort_flag) || !mbar_wait(&c.o_full[0], ic[0] & 1, abort_flag) ||
          (both && !mbar_wait(&c.o_full[1], ic[1] & 1, abort_flag))) {
        ok = false;
        break;
      }
      ++turns;
      tc_fence_after();
      if (r == 0 && w < steps) mbar_arrive(&c.vempty[(tiles + last_v) % kVStages]);
      if (both) {
        const float m0 = c.ml[0][r][0], m1 = c.ml[1][r][0];
        m_ref = fmaxf(m0, m1);
        if (isnan(m0) || isnan(m1)) m_ref = m0 + m1;
        a0 = m0 == -INFINITY ? 0.f : exp2f(m0 - m_ref);
        a1 = m1 == -INFINITY ? 0.f : exp2f(m1 - m_ref);
        l_sum = c.ml[0][r][1] * a0 + c.ml[1][r][1] * a1;
      } else {
        m_ref = c.ml[0][r][0];
        l_sum = c.ml[0][r][1];
      }
    }
    ++ic[0];
    if (both) ++ic[1];
    tiles += info.nt;
    const bool bad = c.bad[slot] != 0, spoilt = *reinterpret_cast<volatile int*>(&c.spoilt[slot]) != 0;
    // columns: a whole row per thread with two row tiles, half of it per stream with one
    const int c0 = two ? 0 : 64 * w;
    uint32_t v[4][32];
    if (two) {
#pragma unroll
      for (int h = 0; h < 4; ++h) tmem_ld32_issue(orow_t + 32 * h, v[h]);
#pragma unroll
      for (int h = 0; h < 4; ++h) tmem_ld32_wait(v[h]);
    } else {
      const uint32_t o0 = tmem + lane_off + kOCol + c0;
      tmem_ld32_issue(o0, v[0]);
      tmem_ld32_issue(o0 + 32, v[1]);
      if (both) {
        tmem_ld32_issue(o0 + 128, v[2]);
        tmem_ld32_issue(o0 + 160, v[3]);
      }
      tmem_ld32_wait(v[0]);
      tmem_ld32_wait(v[1]);
      if (both) {
        tmem_ld32_wait(v[2]);
        tmem_ld32_wait(v[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 32; ++k)
            v[h][k] = __float_as_uint(fmaf(__uint_as_float(v[h][k]), a0, __uint_as_float(v[h + 2][k]) * a1));
      }
    }
    // O is in registers: the next unit's first P V may overwrite it
    tc_fence_before();
    __syncwarp();
    if (lane < 2) {
      if (two) mbar_arrive(&c.o_free[w]);  // (twice per warp: eight arrivals in all)
      else if (lane == 0 || both) mbar_arrive(&c.o_free[lane]);
    }
    const int pieces = two ? 4 : 2;
    if (spoilt && live) {
      // give the values taken out back to the rows that see them (rare)
      const int b0 = max(info.kt0 * kTileKeys, info.ctx), b1 = min((info.kt0 + info.nt) * kTileKeys, info.len);
      for (int u = b0; u < b1; ++u) {
        if (!(seen_bits(mrow, P.mask_words, info.q_len, u - info.ctx) & 1)) continue;
        const int id = __ldg(P.bt + static_cast<int64_t>(info.seq) * P.max_blocks + u / kBlock);
        if (id < 0 || id >= P.num_blocks) continue;
        const __nv_bfloat16* src =
            P.v_cache + ((static_cast<int64_t>(id) * P.hkv + info.head) * kBlock + u % kBlock) * 128 + c0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h >= pieces) break;
          // (32 values at a time, so that v stays in registers)
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float x = __bfloat162float(src[32 * h + k]);
            if (!isfinite(x)) v[h][k] = __float_as_uint(__uint_as_float(v[h][k]) + x);
          }
        }
      }
    }
    if (info.slot >= 0) {
      // the rows' partial: accumulator, then maximum and sum (a sum of -1: a bad block id)
      const int64_t prow = static_cast<int64_t>(info.slot) * P.rows_cap + (two ? 128 * w + r : r);
      if (live) {
        float* dst = P.part_o + prow * 128 + c0;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h >= pieces) break;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t(&w8)[8] = *reinterpret_cast<const uint32_t(*)[8]>(v[h] + 8 * q);
            st_global_v8(dst + 32 * h + 8 * q, w8);
          }
        }
        if (two || w == 0) {
          P.part_ml[prow * 2] = m_ref;
          P.part_ml[prow * 2 + 1] = bad ? -1.f : l_sum;
        }
      }
    } else if (live) {
      const float inv = bad || l_sum == 0.f ? 0.f : 1.f / l_sum;
      const bool zero = bad || l_sum == 0.f;
      __nv_bfloat16* dst = P.out + ((static_cast<int64_t>(info.t0) + j0 + rj) * P.hq +
                                    static_cast<int64_t>(info.head) * P.group + rg) * 128 + c0;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (h >= pieces) break;
        uint32_t wv[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          __nv_bfloat162 h2 =
              __floats2bfloat162_rn(__uint_as_float(v[h][2 * q]) * inv, __uint_as_float(v[h][2 * q + 1]) * inv);
          wv[q] = zero ? 0u : *reinterpret_cast<uint32_t*>(&h2);
        }
        if (P.out_v8) {
#pragma unroll
          for (int q = 0; q < 2; ++q) st_global_v8(dst + 32 * h + 16 * q, *reinterpret_cast<const uint32_t(*)[8]>(wv + 8 * q));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            reinterpret_cast<uint4*>(dst + 32 * h)[q] = make_uint4(wv[4 * q], wv[4 * q + 1], wv[4 * q + 2], wv[4 * q + 3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.item_empty[slot]);
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
}

__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ CUtensorMap qmap,
                                                           const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap, const Params P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // the swizzled tiles need it, and no room is left to round up in
    flag_error(P.err, kErrTimeout);
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
      mbar_init(&c.o_free[w], 8);
      mbar_init(&c.q_full[w], 1);
      mbar_init(&c.q_free[w], 1);
    }
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&c.item_full[s], 1);
      mbar_init(&c.item_empty[s], 9);  // the MMA warp and the eight softmax warps
    }
    mbar_init(&c.joined, 8);
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    c.start_seq = 0;
    c.start_base = 0;
    fence_mbar_init();
    tma_prefetch_map(&qmap);
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  if (warp == 1) tmem_alloc(&c.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  grid_dep_wait();
  grid_dep_launch();
  find_run(P, c);
  if (warp == 0) producer_warp(P, &qmap, &kmap, &vmap, c, qbuf, kbuf, vbuf);
  else if (warp == 1) mma_warp(P, c, qbuf, kbuf, vbuf, tmem);
  else softmax_warps(P, c, vbuf, tmem);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
    tmem_relinquish();
  }
}

// ------------------------------------------------------------------ merge
// One warp per row of a cut unit: the parts' weights 2^(m - M), then the weighted sum of their
// accumulators in the order of the keys.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 32;

__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const Params P) {
  grid_dep_wait();
  grid_dep_launch();
  const int cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4* rec = reinterpret_cast<const int4*>(P.cuts + cta);
  const int4 c0 = __ldcg(rec), c1 = __ldcg(rec + 1);  // parts, head, t0, two; j0[2], nq[2]
  const int parts = c0.x;
  if (parts < 2) return;
  const int row = blockIdx.y * kMergeRows + warp;
  const int w = row >> 7, r = row & 127;
  if (w > c0.w) return;
  const int rj = r >> P.gp_log2, rg = r & (P.gp - 1);
  if (rj >= (w ? c1.w : c1.z) || rg >= P.group) return;
  auto slot_row = [&](int p) -> int64_t {
    return static_cast<int64_t>(p == 0 ? 2 * cta + 1 : 2 * (cta + p)) * P.rows_cap + row;
  };
  float M = -INFINITY;
  bool bad = false, nan = false;
  for (int p = lane; p < parts; p += 32) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(P.part_ml) + slot_row(p));
    nan |= isnan(ml.x);
    M = fmaxf(M, ml.x);
    bad |= ml.y == -1.f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  bad = __any_sync(0xffffffffu, bad);
  if (__any_sync(0xffffffffu, nan)) M = __int_as_float(0x7fffffff);
  float den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < parts; p0 += 32) {
    float weight = 0.f, l = 0.f;
    if (p0 + lane < parts) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(P.part_ml) + slot_row(p0 + lane));
      // (a part without a maximum saw nothing, or nothing but NaN, which its sum says)
      weight = ml.x == -INFINITY ? ml.y * 0.f : exp2f(ml.x - M);
      l = ml.y;
    }
    const int n = min(32, parts - p0);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float a = __shfl_sync(0xffffffffu, weight, p);
      const float lp = __shfl_sync(0xffffffffu, l, p);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(P.part_o + slot_row(p0 + p) * 128) + lane);
      if (a != 0.f) {
        den = fmaf(lp, a, den);
        acc.x = fmaf(o.x, a, acc.x);
        acc.y = fmaf(o.y, a, acc.y);
        acc.z = fmaf(o.z, a, acc.z);
        acc.w = fmaf(o.w, a, acc.w);
      }
    }
  }
  const bool zero = bad || den == 0.f;
  const float inv = zero ? 0.f : 1.f / den;
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 packed = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  if (zero) packed = make_uint2(0, 0);
  const int64_t t = static_cast<int64_t>(c0.z) + (w ? c1.y : c1.x) + rj;
  reinterpret_cast<uint2*>(P.out + (t * P.hq + static_cast<int64_t>(c0.y) * P.group + rg) * 128)[lane] = packed;
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
Layout layout_of(int32_t group, int32_t max_query_len, int ctas) {
  Layout l;
  const int64_t rows = static_cast<int64_t>(max_query_len) << gp_log2_of(group);
  l.rows_cap = static_cast<int>(rows < 256 ? rows : 256);
  const size_t slots = 2 * static_cast<size_t>(ctas) * l.rows_cap;
  l.o_bytes = slots * 128 * sizeof(float);
  l.ml_bytes = (slots * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255);
  l.bytes = l.o_bytes + l.ml_bytes + static_cast<size_t>(ctas) * sizeof(Cut);
  return l;
}

}  // namespace

size_t tree_tc_workspace(int32_t group, int32_t max_query_len, int num_sms) {
  return layout_of(group, max_query_len, num_sms).bytes;
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
  // CTAs: one per SM, fewer where the caller's bounds leave less to do
  const int64_t units = static_cast<int64_t>((a.max_query_len + 2 * p.rows_q - 1) / (2 * p.rows_q)) * hkv;
  const int64_t tiles = units * ((static_cast<int64_t>(a.max_seq_len) + kTileKeys - 1) / kTileKeys);
  const int64_t most = tiles >= num_sms ? num_sms : tiles * a.num_seqs;
  const int ctas = static_cast<int>(most < num_sms ? (most + kMinTiles - 1) / kMinTiles : num_sms);
  const Layout l = layout_of(group, a.max_query_len, num_sms);
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
  p.scale_log2 = a.scale * 1.4426950408889634f;
  static uint64_t smem_set = 0;
  st = set_smem_once(reinterpret_cast<const void*>(tree_kernel), kSmemBytes, &smem_set);
  if (st) return st;
  st = cuda_status(launch_k(tree_kernel, dim3(ctas), dim3(kThreads), kSmemBytes, s, qm, km, vm, p));
  if (st) return st;
  const int row_blocks = (l.rows_cap + kMergeRows - 1) / kMergeRows;
  return cuda_status(launch_k(tree_merge_kernel, dim3(ctas, row_blocks), dim3(kMergeThreads), 0, s, p));
}

}  // namespace pkv
