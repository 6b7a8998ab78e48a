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
//   p = hi + mid / 32 + lo / 1024 of a weight p rounded to fp16 (2^-11); of a small one, below 2^-9, the terms of 2^17 p,
//     in three more columns.  So a weight is held to 2^-11 of itself down to 2^-26, which is 2^-29 of a row's largest weight
//     at least, and smaller ones to 2^-37 (2^-40): a million small weights beside a large one keep their share
//     even where the large one's V is 0.
// Scales: ks multiplies a key's scores.  vs goes into the weight, as log2 vs added to the score, so that a row's
// reference is the largest w vs of it, and out again of the row's sum, which takes p / vs.
// Scores, maxima, sums and accumulators are fp32.
//
// This kernel serves requests of one token: the G query heads of a kv head are the rows, 8 or 16 of them.  (Requests with
// more tokens, and a few single ones beside them: k_q8_chunk.cu.)  A softmax thread is one key of the tile: its
// scales are its own, and its row sums stay in registers until the unit ends.  The reference of a row moves only
// when a score of the tile exceeds it by 2^5, which a vote of the threads tells; only then is a maximum taken
// across them and O rescaled.
//
// Bound: HBM, once the cache is larger than a few MB.  32 requests of 32768 keys, 64 / 8 heads, 2.15 GB: 311 us, 103 % of the measured
// copy rate (DRAM 88 % busy); 64 requests of 128 to 4096 keys, 279 MB: 52 us, 80 %, of which 4 are the start and 4 the
// join; with 128 / 8 heads, 282 MB, 55 us.  The columns of small weights cost none, 0.3 and 1.2 of these.  One request of 500 keys: 8.7 us of latency, 3 of them the join's launch.  Bytes pass through shared memory twice (TMA in,
// the tensor core out); the tensor pipe is 9 % busy.
//
// Per CTA, two to an SM so that one's unit ends while the other streams (192 threads each): warp 0 walks its run
// (q8_units.cuh) and loads K and V by TMA (16 rows of 128 bytes a block, 128-byte swizzle, three tiles in flight), warp 1
// issues the MMAs, the others are softmax.  All waits are bounded.
#include <algorithm>

#include "q8_units.cuh"

namespace pkv {
namespace {

constexpr int kHalfTile = kTileKeys * 128;  // K or V of a tile, bytes
constexpr int kStages = 3, kThreads = 192, kCtasPerSm = 2;
constexpr uint32_t kSCols = 32, kOCol = 64;  // tensor memory: S of even and of odd tiles, O
constexpr int kTerms = 6;                    // of a weight: three, and three for small ones
constexpr float kSmall = 1.f / 512.f, kUp = 131072.f, kDown = 1.f / 131072.f;  // 2^-9, 2^17, 2^-17
constexpr float kTop = 3.f;   // log2 of a row's largest weight when its reference is set
constexpr float kMost = 8.f;  // and the most that it may reach: the rest of a term is then at most 8 units

struct Ctl {
  uint64_t kfull[kStages], vfull[kStages], empty[kStages];
  uint64_t s_full[2], p_full, pv_done, q_full;
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  uint64_t drain;
  Item ring[kItemRing];
  int bad[kItemRing];
  float4 across[16];             // a row's values of the four warps
  float4 moved[4], factor[4];    // how far a row's reference moves, 2^-that
  float reference[16];
  uint32_t largest[4];
  Run<kThreads> run;
  uint32_t tmem_base;
  int abort_flag;
};

template <int kOctets>
struct Shape {
  static constexpr uint32_t kOCols = 8 * kTerms * kOctets, kTmemCols = kOCol + kOCols <= 128 ? 128 : 256;
  static constexpr int kQBytes = 16 * kOctets * 128, kPBytes = 128 * static_cast<int>(kOCols);
  static constexpr int kSmemBytes = kStages * 2 * kHalfTile + kQBytes + kPBytes + static_cast<int>(sizeof(Ctl));
  static_assert(kSmemBytes <= 115712 && kCtasPerSm * kTmemCols <= 512, "two CTAs an SM");
};

__device__ __forceinline__ void raise_abort(Ctl& c, uint32_t* err) {
  *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
  flag_error(err, kErrTimeout);
}

// ------------------------------------------------------------------ producer
__device__ void producer_warp(const Q8Params& P, const CUtensorMap* kmap, const CUtensorMap* vmap, Ctl& c, uint8_t* tiles) {
  const int lane = threadIdx.x & 31, b = lane & 7;
  volatile int* abort_flag = &c.abort_flag;
  Walk walk = start_walk(c.run);
  if (lane < 2) P.cuts[2 * blockIdx.x + lane].parts = 0;
  __syncwarp();
  const bool is_v = lane >= 8;
  const CUtensorMap* map = is_v ? vmap : kmap;
  const uint64_t drop = l2_policy_evict_first();
  uint32_t n = 0, s = 0, phase = 1;
  bool ok = true;
  for (uint32_t it = 0; ok; ++it) {
    const Item item = next_item(P, walk, c.run.len);
    const int slot = it % kItemRing;
    ok = wait_for(&c.item_empty[slot], ((it / kItemRing) & 1) ^ 1, abort_flag);
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
      ok = wait_for(&c.empty[s], phase, abort_flag);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&c.kfull[s], nblk * 2048);
      if (lane == 8) mbar_arrive_expect_tx(&c.vfull[s], nblk * 2048);
      __syncwarp();
      if (lane < 16 && b < nblk)
        tma_load_2d(tiles + s * 2 * kHalfTile + (is_v ? kHalfTile : 0) + b * 2048, map, is_v ? &c.vfull[s] : &c.kfull[s], 0,
                    (cur * P.hkv + item.head) * kBlock, drop);
      ++n;
      if (++s == kStages) {
        s = 0;
        phase ^= 1;
      }
    }
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
  __syncwarp();
  if (*abort_flag) {  // copies already issued land before the CTA's shared memory goes away
#pragma unroll 1
    for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i) {
      wait_for(&c.kfull[i % kStages], (i / kStages) & 1, nullptr);
      wait_for(&c.vfull[i % kStages], (i / kStages) & 1, nullptr);
    }
  }
}

// ------------------------------------------------------------------ MMA warp
// One elected thread issues every MMA; the whole warp walks through the tiles.  A turn is S of the next
// tile, then P V of this one.  MMAs complete in order, and S of tile j + 1 goes over S of tile j - 1, whose weights
// have been handed over by then.
template <int kOctets>
__device__ void mma_warp(const Q8Params& P, Ctl& c, uint32_t tiles, uint32_t qbuf, uint32_t pbuf, uint32_t tmem) {
  constexpr uint32_t s_idesc = umma_idesc_e4m3(128, 16 * kOctets, false, false);
  constexpr uint32_t o_idesc = umma_idesc_e4m3(128, Shape<kOctets>::kOCols, true, true);
  volatile int* abort_flag = &c.abort_flag;
  uint32_t n = 0;  // tiles so far
  bool ok = true, issued = false;
  for (uint32_t it = 0;; ++it) {
    const int slot = it % kItemRing;
    ok = wait_for(&c.item_full[slot], (it / kItemRing) & 1, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const int nt = __shfl_sync(0xffffffffu, c.ring[slot].nt, 0);
    const bool over = __shfl_sync(0xffffffffu, c.ring[slot].idx, 0) < 0;
    __syncwarp();
    if (over) break;
    if (elected()) mbar_arrive(&c.item_empty[slot]);
    ok = wait_for(&c.q_full, it & 1, abort_flag);
    for (int j = -1; j < nt; ++j) {
      // (a wait that is given up may be given up by some lanes only: the warp votes, and goes on together)
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (j + 1 < nt) {
        const uint32_t m = n + j + 1, s = m % kStages;
        ok = wait_for(&c.kfull[s], (m / kStages) & 1, abort_flag);
        tc_fence_after();
        const uint64_t a = umma_smem_desc(tiles + s * 2 * kHalfTile, 16, 1024, kLayout128B);
        const uint64_t b = umma_smem_desc(qbuf, 16, 1024, kLayout128B);
        if (elected()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f8_ss(tmem + (m & 1) * kSCols, umma_desc_advance(a, 32 * k), umma_desc_advance(b, 32 * k), s_idesc, k > 0);
          umma_commit(&c.s_full[m & 1]);
        }
        issued = true;
      }
      if (j < 0) continue;
      const uint32_t m = n + j, s = m % kStages;
      ok = ok && wait_for(&c.vfull[s], (m / kStages) & 1, abort_flag);
      ok = ok && wait_for(&c.p_full, m & 1, abort_flag);
      tc_fence_after();
      const uint64_t a = umma_smem_desc(tiles + s * 2 * kHalfTile + kHalfTile, kHalfTile, 1024, kLayout128B);
      const uint64_t b = umma_smem_desc(pbuf, 128, 2048, kLayoutNone);
      if (elected()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8_ss(tmem + kOCol, umma_desc_advance(a, 4096 * k), umma_desc_advance(b, 512 * k), o_idesc, j > 0 || k > 0);
        umma_commit(&c.pv_done);
        umma_commit(&c.empty[s]);
      }
      issued = true;
    }
    if (!ok) break;
    n += nt;
  }
  if (!ok && !*abort_flag && (threadIdx.x & 31) == 0) raise_abort(c, P.err);
  __syncwarp();
  // every MMA, and the arrivals that its commits trigger, is over before TMEM is freed
  if (issued) {
    if (elected()) umma_commit(&c.drain);
    wait_for(&c.drain, 0, nullptr);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ uint32_t to_e4m3(__half2 x) {
  return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ bool vote(bool x) {  // any of the softmax threads
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void meet() { named_bar_sync(1, 128); }

// One of eight values over the lanes of a warp: lane l gets value l & 7, joined over the warp.
template <typename F>
__device__ __forceinline__ float join8(const Two* y, F&& f) {
  const int lane = threadIdx.x & 31;
  float x[8], a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 z = both(y[i]);
    x[2 * i] = z.x;
    x[2 * i + 1] = z.y;
  }
  const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = f(h4 ? x[i + 4] : x[i], __shfl_xor_sync(0xffffffffu, h4 ? x[i] : x[i + 4], 4));
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = f(h2 ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, h2 ? a[i] : a[i + 2], 2));
  float r = f(h1 ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, h1 ? b[0] : b[1], 1));
  r = f(r, __shfl_xor_sync(0xffffffffu, r, 8));
  return f(r, __shfl_xor_sync(0xffffffffu, r, 16));
}

// (Code that runs once a unit is kept short, in loops: each time it has to be fetched anew.)
template <int kOctets>
__device__ __forceinline__ void softmax_warps(const Q8Params& P, Ctl& c, uint8_t* tiles, uint8_t* q, uint8_t* p, uint32_t tmem) {
  constexpr int kRows = 8 * kOctets, kPairs = kRows / 2;
  constexpr int kPerRow = 128 / 16;  // threads of a row of Q, 16 elements each
  const int lane = threadIdx.x & 31, wq = (threadIdx.x >> 5) & 3;
  const int t = wq * 32 + lane;  // this thread's key of a tile, element of O
  const uint32_t lanes = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  volatile int* abort_flag = &c.abort_flag;
  uint32_t n = 0;        // tiles so far
  float unscale = 0.f;   // of the scores of the unit whose Q is in place: scale log2(e) / c
  bool ok = true;

  // This thread's elements of the unit's rows.
  const auto fetch_q = [&](const Item& item, uint4 (&raw)[2]) {
    const int g = t / kPerRow;
    const uint4* src = reinterpret_cast<const uint4*>(
        P.q + (static_cast<int64_t>(item.t0) * P.hq + static_cast<int64_t>(item.head) * P.group + g) * 128 + t % kPerRow * 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) raw[i] = g < P.group ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  };
  // The rows as e4m3 terms in Q (row r: hi at 16 (r / 8) + r % 8, lo 8 rows further).
  const auto put_q = [&](const uint4 (&raw)[2]) {
    const int r = t / kPerRow, part = t % kPerRow;
    const uint32_t y[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    // the largest finite size: bf16 bits compare as whole numbers
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t a = y[e] & 0x7fffu, b = y[e] >> 16 & 0x7fffu;
      top = max(top, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) c.largest[wq] = top;
    meet();
    top = max(max(c.largest[0], c.largest[1]), max(c.largest[2], c.largest[3]));
    // largest c in [128, 256): a term's rest is at most 8 units, 256 in those of the next
    const int e = max(static_cast<int>(top >> 7) - 127, -119);
    const float up = __int_as_float((127 + 7 - e) << 23);
    unscale = P.scale_log2 * (e >= -100 ? __int_as_float((127 - 7 + e) << 23) : 0.f);
    uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // (times 0 and added: an infinity makes its row NaN)
      float a = __uint_as_float(y[i] << 16), b = __uint_as_float(y[i] & 0xffff0000u);
      a = fmaf(a, up, a * 0.f);
      b = fmaf(b, up, b * 0.f);
      const uint32_t code = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
      const float2 back = __half22float2(from_e4m3(code));
      hi[i / 2] |= code << (16 * (i & 1));
      lo[i / 2] |= static_cast<uint32_t>(
                       __nv_cvt_float2_to_fp8x2(make_float2((a - back.x) * 32.f, (b - back.y) * 32.f), __NV_SATFINITE, __NV_E4M3))
                   << (16 * (i & 1));
    }
    if (r < kRows) {
      const int n_hi = 16 * (r >> 3) + (r & 7);
      uint8_t* to = q + n_hi * 128 + ((part ^ (n_hi & 7)) << 4);
      *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(to + 1024) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.q_full);
  };
  // This thread's block of a tile and its scales.
  const auto id_of = [&](const Item& item, int32_t tile) {
    return __ldg(P.bt + static_cast<int64_t>(item.seq) * P.max_blocks + min(tile * kBlocksPerTile + (t >> 4), (item.len - 1) / kBlock));
  };
  const auto scales_of = [&](const Item& item, int32_t id) {
    return __ldg(P.scales + static_cast<int64_t>(id < 0 || id >= P.num_blocks ? 0 : id) * P.hkv + item.head);
  };

  uint32_t it = 0;
  Item item{};
  // what the next unit begins with: loaded while the last tile of this one is worked on
  uint4 raw[2];
  int32_t id0 = 0, id1 = 0;
  float2 sc = make_float2(0.f, 0.f);
  const auto fetch_unit = [&](const Item& next) {
    fetch_q(next, raw);
    id0 = id_of(next, next.kt0);
    id1 = next.nt > 1 ? id_of(next, next.kt0 + 1) : 0;
  };
  // (the first pass has no unit to work on: it only loads one)
  for (bool first = true; ok; first = false) {
    Two l[kPairs], minus_m[kPairs];
    bool fetched = false;
    if (!first) {
      const int32_t tile_end = item.kt0 + item.nt;
      const float factor = unscale;
      int32_t id = id1;
#pragma unroll
      for (int r = 0; r < kPairs; ++r) minus_m[r] = l[r] = two(0.f);
#pragma unroll 1
      for (int j = 0; j < item.nt; ++j, ++n) {
        const int32_t tile = item.kt0 + j;
        const float2 now = sc;
        if (tile + 1 < tile_end) {
          sc = scales_of(item, id);
          if (tile + 2 < tile_end) id = id_of(item, tile + 2);
        } else if (mbar_test(&c.item_full[(it + 1) % kItemRing], ((it + 1) / kItemRing) & 1)) {
          fetched = true;
          const Item& next = c.ring[(it + 1) % kItemRing];
          if (next.idx >= 0) fetch_unit(next);
        }
        const float ks = now.x * factor, lv = __log2f(fminf(fmaxf(now.y, kLeastV), kMostV)), iv = ex2_approx(-lv);
        ok = wait_for(&c.s_full[n & 1], (n >> 1) & 1, abort_flag);
        tc_fence_after();
        // Keys behind the context have no weight, and V no values there (a weight of 0 times a NaN is one).
        const bool edge = (tile + 1) * kTileKeys > item.len, hidden = edge && tile * kTileKeys + t >= item.len;
        if (edge) {
          ok = ok && wait_for(&c.vfull[n % kStages], (n / kStages) & 1, abort_flag);
          if (hidden && ok) {
            uint4* row = reinterpret_cast<uint4*>(tiles + n % kStages * 2 * kHalfTile + kHalfTile + t * 128);
#pragma unroll 1
            for (int ch = 0; ch < 8; ++ch) row[(ch + t) & 7] = make_uint4(0, 0, 0, 0);
          }
        }
        Two x[kPairs];
        float most = -INFINITY;
        uint32_t v[kOctets][16];
#pragma unroll
        for (int g = 0; g < kOctets; ++g) tmem_ld16_sync(lanes + (n & 1) * kSCols + 16 * g, v[g]);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const uint32_t* y = v[i / 4] + 2 * (i % 4);
          const Two hi = two(__uint_as_float(y[0]), __uint_as_float(y[1])), lo = two(__uint_as_float(y[8]), __uint_as_float(y[9]));
          x[i] = add2(fma2(fma2(lo, two(1.f / 32.f), hi), two(ks), two(lv)), minus_m[i]);
          if (hidden) x[i] = two(-INFINITY);
          const float2 z = both(x[i]);
          most = fmaxf(most, fmaxf(z.x, z.y));
        }
        // the place of the weights is free again when the products with those before have been made
        if (j > 0) ok = ok && wait_for(&c.pv_done, (n - 1) & 1, abort_flag);
        // (every run has a visible key in its first tile: each row gets its reference there)
        if (vote(most > kMost || j == 0 || !ok)) {
          if (vote(!ok)) {  // (a wait that some thread gave up ends here for all of them)
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kOctets; ++g) {
            const float top = join8(x + 4 * g, [](float a, float b) { return fmaxf(a, b); });
            if (lane < 8) reinterpret_cast<float*>(&c.across[8 * g + lane])[wq] = top;
          }
          meet();
          if (t < kRows) {
            const float4 y = c.across[t];
            const float top = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));  // (NaN is passed over)
            const float more = j > 0 ? fmaxf(top - kTop, 0.f) : top > -INFINITY ? top - kTop : 0.f;
            reinterpret_cast<float*>(c.moved)[t] = -more;
            reinterpret_cast<float*>(c.factor)[t] = j > 0 ? ex2_approx(-more) : 1.f;  // (nothing is summed up before the first)
          }
          meet();
#pragma unroll
          for (int i = 0; i < kRows / 4; ++i) {
            const float4 d = c.moved[i], f = c.factor[i];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const Two m = h ? two(d.z, d.w) : two(d.x, d.y);
              x[2 * i + h] = add2(x[2 * i + h], m);
              minus_m[2 * i + h] = add2(minus_m[2 * i + h], m);
              l[2 * i + h] = mul2(l[2 * i + h], h ? two(f.z, f.w) : two(f.x, f.y));
            }
          }
          if (j > 0) {
#pragma unroll 1
            for (int k = 0; k < kTerms * kOctets; ++k) {
              const float4 f0 = c.factor[k / kTerms * 2], f1 = c.factor[k / kTerms * 2 + 1];
              const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
              uint32_t o[8];
              tmem_ld8_sync(lanes + kOCol + 8 * k, o);
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
              tmem_st8(lanes + kOCol + 8 * k, o);
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int g = 0; g < kOctets; ++g) {
          uint32_t b[3][2] = {}, small[2] = {};  // (all ones: of a small weight)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 z = both(x[4 * g + e]);
            const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
            l[4 * g + e] = fma2(two(p0, p1), two(iv), l[4 * g + e]);
            const bool small0 = p0 < kSmall, small1 = p1 < kSmall;
            small[e / 2] |= ((small0 ? 0xffu : 0u) | (small1 ? 0xff00u : 0u)) << (16 * (e & 1));
            const __half2 y = __floats2half2_rn(p0 * (small0 ? kUp : 1.f), p1 * (small1 ? kUp : 1.f));
            const uint32_t hi = to_e4m3(y);
            const __half2 y1 = __hmul2(__hsub2(y, from_e4m3(hi)), __float2half2_rn(32.f));
            const uint32_t mid = to_e4m3(y1);
            const __half2 y2 = __hmul2(__hsub2(y1, from_e4m3(mid)), __float2half2_rn(32.f));
            b[0][e / 2] |= hi << (16 * (e & 1));
            b[1][e / 2] |= mid << (16 * (e & 1));
            b[2][e / 2] |= to_e4m3(y2) << (16 * (e & 1));
          }
          // eight columns a term: those of weights that are not small, then of those that are
          uint4* to = reinterpret_cast<uint4*>(p + kTerms / 2 * g * 2048 + t * 16);
          const uint32_t s0 = small[0], s1 = small[1];
          to[0] = make_uint4(b[0][0] & ~s0, b[0][1] & ~s1, b[1][0] & ~s0, b[1][1] & ~s1);
          to[128] = make_uint4(b[2][0] & ~s0, b[2][1] & ~s1, b[0][0] & s0, b[0][1] & s1);
          to[256] = make_uint4(b[1][0] & s0, b[1][1] & s1, b[2][0] & s0, b[2][1] & s1);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.p_full);
      }
      if (!ok) break;
    }
    // the next unit's rows, while the last products run
    const uint32_t at = first ? it : it + 1;
    ok = wait_for(&c.item_full[at % kItemRing], (at / kItemRing) & 1, abort_flag);
    ok = !vote(!ok);  // (what follows has barriers: all threads go on, or none)
    if (!ok) break;
    const Item next = c.ring[at % kItemRing];
    if (next.idx >= 0) {
      if (!fetched) fetch_unit(next);
      sc = scales_of(next, id0);
      put_q(raw);
    }
    if (!first) {
#pragma unroll
      for (int g = 0; g < kOctets; ++g) {
        const float sum = join8(l + 4 * g, [](float a, float b) { return a + b; });
        if (lane < 8) reinterpret_cast<float*>(&c.across[8 * g + lane])[wq] = sum;
      }
      if (item.slot >= 0 && t == 0) {
#pragma unroll
        for (int r = 0; r < kPairs; ++r) {
          const float2 m = both(minus_m[r]);
          c.reference[2 * r] = -m.x;
          c.reference[2 * r + 1] = -m.y;
        }
      }
      ok = wait_for(&c.pv_done, (n - 1) & 1, abort_flag);
      ok = !vote(!ok);
      if (!ok) break;
      tc_fence_after();
      const bool bad = *reinterpret_cast<volatile int*>(&c.bad[it % kItemRing]) != 0;
      __nv_bfloat16* out = P.out + (static_cast<int64_t>(item.t0) * P.hq + static_cast<int64_t>(item.head) * P.group) * 128 + t;
#pragma unroll 1
      for (int g = 0; g < kOctets; ++g) {
        uint32_t v[kTerms][8];
#pragma unroll
        for (int k = 0; k < kTerms; ++k) tmem_ld8_sync(lanes + kOCol + 8 * (kTerms * g + k), v[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 8 * g + e;
          const float4 y = c.across[r];
          const float sum = (y.x + y.y) + (y.z + y.w);
          const auto sum_of = [&](int k) {
            return fmaf(__uint_as_float(v[k + 2][e]), 1.f / 1024.f, fmaf(__uint_as_float(v[k + 1][e]), 1.f / 32.f, __uint_as_float(v[k][e])));
          };
          const float o = fmaf(sum_of(3), kDown, sum_of(0));
          if (r < P.group) {
            if (item.slot >= 0) {
              const int64_t row = static_cast<int64_t>(item.slot) * P.rows_cap + r;
              P.part_o[row * 128 + t] = o;
              if (t == 0) {
                // (of a row that saw nothing, or a NaN, the sum says it all)
                P.part_ml[2 * row] = sum != 0.f && sum == sum ? c.reference[r] : -INFINITY;
                P.part_ml[2 * row + 1] = bad ? -1.f : sum;
              }
            } else {
              out[r * 128] = __float2bfloat16_rn(bad || sum == 0.f ? 0.f : __fdividef(o, sum));
            }
          }
        }
      }
      tc_fence_before();
      meet();  // O and the sums have been read
      if (t == 0) mbar_arrive(&c.item_empty[it % kItemRing]);
    }
    if (next.idx < 0) break;
    it = at;
    item = next;
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
}

template <int kOctets>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Q8Params P) {
  using S = Shape<kOctets>;
  extern __shared__ __align__(1024) uint8_t tiles[];
  uint8_t* qbuf = tiles + kStages * 2 * kHalfTile;
  uint8_t* pbuf = qbuf + S::kQBytes;
  Ctl& c = *reinterpret_cast<Ctl*>(pbuf + S::kPBytes);
  const int warp = threadIdx.x >> 5;
  if ((smem_u32(tiles) & 1023u) != 0) {  // (there is no room to move up; swizzled tiles would not be where they are looked for)
    grid_dep_wait();
    if (threadIdx.x == 0) flag_error(P.err, kErrTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&c.kfull[s], 1);
      mbar_init(&c.vfull[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    mbar_init(&c.s_full[0], 1);
    mbar_init(&c.s_full[1], 1);
    mbar_init(&c.p_full, 4);
    mbar_init(&c.pv_done, 1);
    mbar_init(&c.q_full, 4);
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(&c.item_full[s], 1);
      mbar_init(&c.item_empty[s], 2);  // MMA warp, softmax
    }
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem_base, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  grid_dep_wait();
  grid_dep_launch();
  find_run(P, c.run);
  if (warp == 0) producer_warp(P, &kmap, &vmap, c, tiles);
  else if (warp == 1) mma_warp<kOctets>(P, c, smem_u32(tiles), smem_u32(qbuf), smem_u32(pbuf), tmem);
  else softmax_warps<kOctets>(P, c, tiles, qbuf, pbuf, tmem);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// The partials of one kernel, and of the other from slot `first` on.
struct Partials {
  const Cut* cuts;
  const float *o, *ml;
  int rows_cap;
};
__global__ void __launch_bounds__(kMergeThreads) q8_merge_kernel(const Q8Params P, const Partials one, const Partials other, int first) {
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  const int at_slot = static_cast<int>(blockIdx.x);
  const bool is_other = at_slot >= first;
  join_rows<4>(
      is_other ? other.cuts : one.cuts, is_other ? other.o : one.o, is_other ? other.ml : one.ml, is_other ? other.rows_cap : one.rows_cap,
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
      },
      is_other ? at_slot - first : at_slot, is_other ? static_cast<int>(gridDim.x) - first : first);
}

int gp_log2_of(int group) {
  int g = 0;
  while ((1 << g) < group) ++g;
  return g;
}

// The partials of a kernel: the one of this file (`single`), or that of k_q8_chunk.cu.
struct Layout {
  int rows_cap, runs;
  size_t o_bytes, ml_bytes, bytes;
};
Layout layout_of(bool single, int32_t group, int32_t max_query_len, int num_sms) {
  Layout l;
  const int64_t rows = static_cast<int64_t>(single ? 1 : max_query_len) << gp_log2_of(group);
  l.rows_cap = static_cast<int>(rows < 256 ? rows : 256);
  l.runs = single ? num_sms * kCtasPerSm : num_sms;
  const size_t slots = 2 * static_cast<size_t>(l.runs) * l.rows_cap;
  l.o_bytes = slots * 128 * sizeof(float);
  l.ml_bytes = (slots * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255);
  l.bytes = (l.o_bytes + l.ml_bytes + 2 * l.runs * sizeof(Cut) + 255) & ~static_cast<size_t>(255);
  return l;
}

template <int kOctets>
int launch_single(const AttnArgs& a, const Q8Params& p, uint64_t rows, int ctas, cudaStream_t s) {
  CUtensorMap km, vm;  // (rows of 128 bytes)
  int st = encode_tensor_map_2d(&km, a.k_cache, 64, rows, 128, 64, 16);
  if (!st) st = encode_tensor_map_2d(&vm, a.v_cache, 64, rows, 128, 64, 16);
  static uint64_t smem_set = 0;
  constexpr int kBytes = Shape<kOctets>::kSmemBytes;
  if (!st) st = set_smem_once(reinterpret_cast<const void*>(q8_kernel<kOctets>), kBytes, &smem_set);
  return st ? st : cuda_status(launch_k(q8_kernel<kOctets>, dim3(ctas), dim3(kThreads), kBytes, s, km, vm, p));
}

}  // namespace

size_t q8_workspace(const pkv_cache_desc& c, int32_t num_q_heads, int32_t max_query_len, int num_sms) {
  const int32_t group = num_q_heads / c.num_kv_heads;
  return layout_of(true, group, max_query_len, num_sms).bytes +
         (max_query_len > 1 ? layout_of(false, group, max_query_len, num_sms).bytes : 0);
}

int launch_q8(const AttnArgs& a, const float* scales, void* workspace, int num_sms, uint32_t* err, cudaStream_t s) {
  const int hkv = a.cache.num_kv_heads, group = a.num_q_heads / hkv;
  const uint64_t rows = static_cast<uint64_t>(a.cache.num_blocks) * hkv * kBlock;
  if (rows >= (1ull << 31)) return PKV_ERR_UNSUPPORTED;
  Q8Params p{};
  p.gp_log2 = gp_log2_of(group);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.scales = reinterpret_cast<const float2*>(scales);
  p.bt = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out_v8 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0 ? 1 : 0;
  p.err = err;
  p.num_blocks = a.cache.num_blocks;
  p.num_tokens = a.num_tokens;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.max_q = a.max_query_len;
  p.hkv = hkv;
  p.hq = a.num_q_heads;
  p.group = group;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  // Steps of single tokens take the kernel of this file, others that of k_q8_chunk.cu, and where many requests must be, or are likely
  // to be, of one token beside longer ones, each kernel takes its own.  One kernel and two: 256 requests of 500 to 3000 keys beside 2 chunks
  // of 512 465 and 197 us, 100 beside 8 288 and 188, 16 beside one 52 and 49; 64 requests of 30 tokens 87 and 96, of 5 79 and 84,
  // 8 of 16 24 and 29
  const bool single = a.max_query_len == 1;
  const bool both = !single && (a.num_tokens < 2 * static_cast<int64_t>(a.num_seqs) ||
                                static_cast<int64_t>(a.max_query_len) * a.num_seqs >= 4 * a.num_tokens);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  Partials parts[2] = {};
  int ctas[2] = {0, 0};
  for (int k = 0; k < 2; ++k) {  // single tokens, chunks
    if (k == 0 ? !single && !both : single) continue;
    const Layout l = layout_of(k == 0, group, a.max_query_len, num_sms);
    Q8Params x = p;
    x.unit_q_log2 = k == 0 ? 0 : 8 - p.gp_log2;
    x.least_q = k == 1 && both ? 2 : 1;
    x.most_q = k == 0 ? 1 : a.max_query_len;
    x.reports = k == 0 || !both;
    // CTAs: all that fit, fewer where the caller's bounds leave less to do
    const int64_t units = (((static_cast<int64_t>(x.most_q) - 1) >> x.unit_q_log2) + 1) * hkv;
    const int64_t key_tiles = (static_cast<int64_t>(a.max_seq_len) + kTileKeys - 1) / kTileKeys;
    const int64_t tiles = units >= l.runs ? units : units * key_tiles;  // (enough to know)
    const int64_t most = tiles >= l.runs ? tiles : tiles * a.num_seqs;
    ctas[k] = static_cast<int>(most < l.runs ? most : l.runs);
    // (a unit's beginning and end as key tiles.  8 requests of 512 tokens: 118.9, 118.5, 118.9, 120.1 us with 2, 3, 4, 5; 33 of 1 to 61:
    // 34.3, 35.5, 36.9, 38.3; 64 of 30: 88.5, 87.8, 86.3, 87.5.  Single tokens: no difference)
    x.unit_cost = most < l.runs ? 0 : 2;
    x.min_run = 1 + x.unit_cost;
    x.rows_cap = l.rows_cap;
    x.part_o = reinterpret_cast<float*>(at);
    x.part_ml = reinterpret_cast<float*>(at + l.o_bytes);
    x.cuts = reinterpret_cast<Cut*>(at + l.o_bytes + l.ml_bytes);
    parts[k] = Partials{x.cuts, x.part_o, x.part_ml, l.rows_cap};
    at += l.bytes;
    const int st = k == 1 ? launch_q8_chunks(x, ctas[k], s) : group > 8 ? launch_single<2>(a, x, rows, ctas[k], s) : launch_single<1>(a, x, rows, ctas[k], s);
    if (st) return st;
  }
  const unsigned rows_ctas = std::max(merge_ctas(parts[0].rows_cap), merge_ctas(parts[1].rows_cap));
  return cuda_status(launch_k(q8_merge_kernel, dim3(2 * (ctas[0] + ctas[1]), rows_ctas), dim3(kMergeThreads), 0, s, p, parts[0], parts[1],
                              2 * ctas[0]));
}

}  // namespace pkv
