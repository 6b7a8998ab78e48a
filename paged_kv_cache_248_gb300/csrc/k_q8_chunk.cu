// k_q8_chunk.cu -- attention of chunks (requests with several tokens) over a paged cache in 8 bits, on
// tcgen05 tensor cores.
//
// Mathematics.  out = sum_u softmax_u(scale q.K_u) V_u with K_u = ks code_u, V_u = vs code_u, over the keys up to a row's
// own token, in one pass over the keys with a running maximum and sum per row.  Tiles of codes become fp16 in shared
// memory, which is exact (e4m3 has 4 significant bits and exponents from -9 to 8); Q becomes fp16 times a
// power of two for each 32 rows, exact down to 2^-24 of their largest element.  A block's scales
// meet the scores: score * ks + log2 vs, so that a row's reference is the largest w vs of it, and its sum takes p / vs.
// The weights are rounded to fp16 (2^-11 of each); they reach 2^7 when a reference is set and 2^15 at most, so that those of
// 2^-21 of the largest and more keep all of their digits.
//
// Why conversion here and not in k_q8.cu: a tile is shared by up to 256 rows, so that converting it costs less
// than splitting every row's weights into 8-bit terms (8 requests of 512 tokens: 337 us with 8-bit products).
//
// Rows.  The G query heads of a kv head are folded into the 128 rows of an MMA tile, 128 / GP tokens by GP heads (GP = G
// rounded up to a power of two).  A unit (q8_units.cuh) is (request, kv head, up to two row tiles), whose key tiles are
// loaded and converted once.
//
// Per CTA (448 threads): warp 0 walks the run, warp 1 issues the MMAs, warps 2-5 and 6-9 are the softmax of a row tile each
// (a thread a row; P stays in tensor memory, over S), warps 10-13 load codes from the cache, 16 bytes a lane and a tile
// ahead in registers, convert them and put them into the K and V rings (two tiles each, 128-byte swizzle).  The row tiles
// take turns: one's products are made while the other's weights are.
// The reference of a row is set by its first tile and moves only when a weight would pass 2^15, which a vote of the warp tells
// as the weights are made: one pass over S (with a pass for the maximum before it 122 us, so 117).
//
// Bound: the chain S (800 clocks with its latency) -> weights (1900) -> P V (500) of a row tile, two of which take turns: 3850 for a
// key tile of 256 rows, where the tensor core is at work for 2100.  8 requests of 512 tokens, contexts of 0 to 2048, 32 / 8 heads:
// 117 us, 735 TFLOP/s, 38 % of cuBLAS's burst; 105 of it here, 12 joining.  A unit's beginning and end cost 7000
// clocks, most of them Q's way to shared memory and O's out of tensor memory.
//
// V rows behind the context are zero; in a tile that not every row sees whole, NaN codes of V are taken out and
// told to the softmax, which makes the rows that see them NaN.  All waits are bounded.
#include "q8_units.cuh"
#include "softmax_row.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 448;
constexpr int kHalfBytes = 16384;
constexpr int kTileBytes = 2 * kHalfBytes;  // 128 x 128 fp16 in two 64-column halves
constexpr int kStages = 2;                  // of K, and of V
constexpr uint32_t kTmemCols = 512;         // S_0, S_1 (P over their first 64 columns), O_0, O_1
constexpr uint32_t kOCol = 256;
constexpr float kTop = 7.f;   // log2 of a row's largest weight when its reference is set
constexpr float kMost = 8.f;  // how much more a weight may be before the reference moves

// Of a key tile (by number, four of them): its blocks' scales, and the keys whose V held a NaN.
struct TileInfo {
  float ks[8], lv[8], iv[8];
  uint32_t spoilt[4];
};

struct Ctl {
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t s_full[2], o_full[2], o_free[2], p_full[2], q_full[2];
  uint64_t item_full[kItemRing], item_empty[kItemRing];
  uint64_t drain;
  Item ring[kItemRing];
  int bad[kItemRing];
  TileInfo info[4];
  Run<kThreads> run;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr int kSmemBytes = (2 + 2 * kStages) * kTileBytes + static_cast<int>(sizeof(Ctl)) + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of the chunk attention");

__device__ __forceinline__ void raise_abort(Ctl& c, uint32_t* err) {
  *reinterpret_cast<volatile int*>(&c.abort_flag) = 1;
  flag_error(err, kErrTimeout);
}

// Tokens of row tile w of an item.
__device__ __forceinline__ int tokens_of(const Q8Params& P, int nq, int w) {
  const int all = 128 >> P.gp_log2;
  return max(0, min(all, nq - w * all));
}

// ------------------------------------------------------------------ walk
__device__ void walk_warp(const Q8Params& P, Ctl& c) {
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &c.abort_flag;
  Walk walk = start_walk(c.run);
  if (lane < 2) P.cuts[2 * blockIdx.x + lane].parts = 0;
  __syncwarp();
  bool ok = true;
  for (uint32_t it = 0;; ++it) {
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
    // the rows of Q on their way to L2: a token's heads are contiguous
    const int bytes = P.group * 256;
    for (int at = lane * 128; at < item.nq * bytes; at += 32 * 128) {
      const int j = at / bytes;
      const char* p = reinterpret_cast<const char*>(P.q + ((static_cast<int64_t>(item.t0) + item.j0 + j) * P.hq +
                                                           static_cast<int64_t>(item.head) * P.group) * 128) + (at - j * bytes);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    }
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
  __syncwarp();
}

// ------------------------------------------------------------------ conversion
// A converter's place in the run: its item, and the tile that it loads next.
struct Cursor {
  Item item;
  uint32_t it;
  int32_t tile, end;
};

// Two fp16 of the pair of codes in the lower half of x.
__device__ __forceinline__ uint32_t halves(uint32_t x) {
  const __half2 h = from_e4m3(x & 0xffffu);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Warp w of four loads blocks 2 w and 2 w + 1 of a tile: rows i * 4 + lane / 8 of each, 16 codes a lane.
__device__ void convert_warps(const Q8Params& P, Ctl& c, uint8_t* kbuf, uint8_t* vbuf) {
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 10;
  const int chunk = lane & 7, sub = lane >> 3;
  volatile int* abort_flag = &c.abort_flag;
  Cursor next{};
  next.item.idx = -1;
  bool ok = true;
  // the two blocks' ids of the tile that is loaded next, and what has been loaded of the one after the present
  int32_t id[2] = {0, 0};
  uint4 kraw[8], vraw[8];
  float2 sc[2];
  // Goes on to the next tile (waiting for its item), false: there is none.
  const auto advance = [&](bool begin) {
    if (!begin && ++next.tile < next.end) return true;
    if (!begin) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.item_empty[next.it % kItemRing]);
      ++next.it;
    }
    ok = ok && wait_for(&c.item_full[next.it % kItemRing], (next.it / kItemRing) & 1, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    next.item = c.ring[next.it % kItemRing];
    __syncwarp();
    next.tile = next.item.kt0;
    next.end = next.item.kt0 + next.item.nt;
    return next.item.idx >= 0;
  };
  const auto ids = [&]() {
    const int32_t last = (next.item.len - 1) / kBlock;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int32_t at = next.tile * kBlocksPerTile + 2 * w + b;
      id[b] = at <= last ? __ldg(P.bt + static_cast<int64_t>(next.item.seq) * P.max_blocks + at) : -1;
      if (at <= last && (id[b] < 0 || id[b] >= P.num_blocks)) {
        if (lane == 0) {
          flag_error(P.err, kErrBlockId);
          *reinterpret_cast<volatile int*>(&c.bad[next.it % kItemRing]) = 1;
        }
        id[b] = -1;
      }
    }
  };
  const auto load = [&](const uint8_t* cache, uint4 (&raw)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t from = id[i / 4];
      raw[i] = make_uint4(0, 0, 0, 0);
      if (from >= 0)
        raw[i] = __ldg(reinterpret_cast<const uint4*>(cache + (static_cast<int64_t>(from) * P.hkv + next.item.head) * (kBlock * 128)) +
                       (i & 3) * 32 + lane);
    }
  };
  const auto store = [&](uint8_t* tile, int i, const uint4& raw) {
    const int row = 32 * w + (i / 4) * kBlock + (i & 3) * 4 + sub;
    const uint4 a = make_uint4(halves(raw.x), halves(raw.x >> 16), halves(raw.y), halves(raw.y >> 16));
    const uint4 b = make_uint4(halves(raw.z), halves(raw.z >> 16), halves(raw.w), halves(raw.w >> 16));
    // 16 values are two chunks of a row of a half tile; lanes of the upper half begin with the second one, so that eight
    // lanes cover all banks
    uint8_t* to = tile + (chunk >> 2) * kHalfBytes + row * 128;
    const int ch = (chunk & 3) * 2, second = chunk >> 2;
    *reinterpret_cast<uint4*>(to + (((ch + second) ^ (row & 7)) << 4)) = second ? b : a;
    *reinterpret_cast<uint4*>(to + (((ch + 1 - second) ^ (row & 7)) << 4)) = second ? a : b;
  };
  bool more = advance(true);
  if (more) {
    ids();
    load(P.k_cache, kraw);
    load(P.v_cache, vraw);
#pragma unroll
    for (int b = 0; b < 2; ++b) sc[b] = __ldg(P.scales + static_cast<int64_t>(max(id[b], 0)) * P.hkv + next.item.head);
  }
  for (uint32_t n = 0; more; ++n) {
    const uint32_t s = n % kStages, phase = ((n / kStages) & 1) ^ 1;
    const int32_t k0 = next.tile * kTileKeys, len = next.item.len;
    const bool edge = k0 + kTileKeys > next.item.ctx + next.item.j0 + 1;
    float2 now[2] = {sc[0], sc[1]};
    ok = ok && wait_for(&c.kempty[s], phase, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    TileInfo& info = c.info[n & 3];
    if (lane < 2) {
      const float2 x = lane ? now[1] : now[0];
      const float lv = __log2f(fminf(fmaxf(x.y, kLeastV), kMostV));
      info.ks[2 * w + lane] = x.x;
      info.lv[2 * w + lane] = lv;
      info.iv[2 * w + lane] = ex2_approx(-lv);
    }
    if (lane == 2) info.spoilt[w] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) store(kbuf + s * kTileBytes, i, kraw[i]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.kfull[s]);
    more = advance(false);
    if (!ok) break;
    if (more) {
      ids();
      load(P.k_cache, kraw);
    }
    ok = wait_for(&c.vempty[s], phase, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    if (edge) {
      uint32_t found = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (i / 4) * kBlock + (i & 3) * 4 + sub;
        const bool past = k0 + 32 * w + row >= len;
        const bool nan = !past && (nan_codes(vraw[i].x) | nan_codes(vraw[i].y) | nan_codes(vraw[i].z) | nan_codes(vraw[i].w)) != 0;
        if (nan) found |= 1u << row;
        if (past || nan) vraw[i] = make_uint4(0, 0, 0, 0);
      }
      found = __reduce_or_sync(0xffffffffu, found);
      if (lane == 0) info.spoilt[w] = found;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) store(vbuf + s * kTileBytes, i, vraw[i]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.vfull[s]);
    if (more) {
      load(P.v_cache, vraw);
#pragma unroll
      for (int b = 0; b < 2; ++b) sc[b] = __ldg(P.scales + static_cast<int64_t>(max(id[b], 0)) * P.hkv + next.item.head);
    }
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
  __syncwarp();
}

// ------------------------------------------------------------------ MMA warp
// 32-bit instruction descriptor for kind::f16 with fp16 A/B (format code 0) and an f32 accumulator.
__device__ constexpr uint32_t idesc_f16(bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

// One elected thread issues every MMA, but the whole warp walks through the tiles, the row tiles in turn: one's products are
// made while the other's weights are.  A row tile's step is P V of its key tile before, then S of its next one: MMAs of
// one thread complete in order, so S cannot overwrite the P that this P V reads, and S being complete tells the softmax that O
// holds every tile before.
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

  // O_w += P_w V of tile number n; `first` begins O_w anew, `last` reports it, `frees`: V has been read.
  __device__ __forceinline__ void pv(int w, uint32_t n, bool first, bool last, bool frees) {
    const uint32_t slot = n & 1, s_col = tmem + 128 * w;
    const uint64_t b = umma_smem_desc(v + slot * kTileBytes, kHalfBytes, 1024, kLayout128B);
    wait(&c.vfull[slot], n >> 1 & 1);
    if (first) {
      wait(&c.o_free[w], (o_phase >> w & 1) ^ 1);
      o_phase ^= 1u << w;
    }
    wait(&c.p_full[w], p_phase >> w & 1);
    p_phase ^= 1u << w;
    tc_fence_after();
    if (elected()) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_f16_ts(s_col + kOCol, s_col + 8 * kk, umma_desc_advance(b, kk * 2048), idesc_f16(true), (!first || kk > 0) ? 1u : 0u);
      if (frees) umma_commit(&c.vempty[slot]);
      if (last) umma_commit(&c.o_full[w]);
    }
  }

  // S_w = Q_w K^T of tile number n; `frees`: K has been read.
  __device__ __forceinline__ void s(int w, uint32_t n, bool frees) {
    const uint32_t slot = n & 1;
    const uint64_t a = umma_smem_desc(q + w * kTileBytes, 16, 1024, kLayout128B);
    const uint64_t b = umma_smem_desc(k + slot * kTileBytes, 16, 1024, kLayout128B);
    wait(&c.kfull[slot], n >> 1 & 1);
    tc_fence_after();
    if (elected()) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t off = h * kHalfBytes + kk * 32;
          umma_f16_ss(tmem + 128 * w, umma_desc_advance(a, off), umma_desc_advance(b, off), idesc_f16(false), h + kk > 0);
        }
      }
      umma_commit(&c.s_full[w]);
      if (frees) umma_commit(&c.kempty[slot]);
    }
    issued = true;
  }

  __device__ __forceinline__ void q_ready(int w) {
    wait(&c.q_full[w], q_phase >> w & 1);
    q_phase ^= 1u << w;
  }
};

__device__ void mma_warp(const Q8Params& P, Ctl& c, uint8_t* qbuf, uint8_t* kbuf, uint8_t* vbuf, uint32_t tmem) {
  static_assert(kStages == 2, "a tile's slot is its number's lowest bit");
  volatile int* abort_flag = &c.abort_flag;
  Issuer x{c, tmem, smem_u32(qbuf), smem_u32(kbuf), smem_u32(vbuf), abort_flag, 0, 0, 0, false, false};
  uint32_t n = 0;  // tiles
  bool ok = true;
  for (uint32_t it = 0; ok; ++it) {
    const int slot = it % kItemRing;
    x.wait(&c.item_full[slot], (it / kItemRing) & 1);
    ok = x.ok();
    if (!ok) break;
    const int nt = __shfl_sync(0xffffffffu, c.ring[slot].nt, 0);
    const int rows = tokens_of(P, __shfl_sync(0xffffffffu, c.ring[slot].nq, 0), 1) > 0 ? 2 : 1;
    const bool over = __shfl_sync(0xffffffffu, c.ring[slot].idx, 0) < 0;
    __syncwarp();
    if (over) break;
    if (elected()) mbar_arrive(&c.item_empty[slot]);
    // turns of the row tiles: 0, 1, 0, 1, ... (one row tile: 0, 0, ...)
    int w = 0;
#pragma unroll 1
    for (int j = 0; j <= nt && ok;) {
      if (j == 0) x.q_ready(w);
      if (j > 0) x.pv(w, n + j - 1, j == 1, j == nt, w == rows - 1);
      if (j < nt) x.s(w, n + j, w == rows - 1);
      ok = x.ok();
      if (++w == rows) {
        w = 0;
        ++j;
      }
    }
    n += nt;
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

// ------------------------------------------------------------------ softmax
// (A warp goes on, or gives up, together.)
__device__ __forceinline__ bool all(bool x) { return __all_sync(0xffffffffu, x) != 0; }

// The largest of 16 scores of a block; with kMask, the first nvis of them count.
template <bool kMask>
__device__ __forceinline__ float largest16(const uint32_t* s, int nvis) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const float a = !kMask || k < nvis ? __uint_as_float(s[k]) : -INFINITY;
    const float b = !kMask || k + 1 < nvis ? __uint_as_float(s[k + 1]) : -INFINITY;
    m[k / 2 & 3] = fmax3(m[k / 2 & 3], a, b);
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The largest score * ks + log2 vs of a row's 128 (the first nvis), two blocks at a time.
template <bool kMask>
__device__ __forceinline__ float row_largest(uint32_t taddr, const TileInfo& info, float factor, int nvis) {
  float top = -INFINITY;
  uint32_t a[32];
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    if (kMask && !__any_sync(0xffffffffu, nvis > 32 * h)) break;  // (no row of the warp sees more)
    tmem_ld32_issue(taddr + 32 * h, a);
    tmem_ld32_wait(a);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float m = largest16<kMask>(a + 16 * b, nvis - 32 * h - 16 * b);
      // (no key of the block: -inf, whatever its scales are)
      const float x = fmaf(m, factor * info.ks[2 * h + b], info.lv[2 * h + b]);
      top = fmaxf(top, !kMask || nvis > 32 * h + 16 * b ? x : -INFINITY);
    }
  }
  return top;
}

// Multiplies a row's O, or `pieces` of 32 fp16 weights, by alpha.
__device__ __forceinline__ void scale_o(uint32_t taddr, float alpha) {
#pragma unroll 1
  for (int ch = 0; ch < 8; ++ch) {
    uint32_t v[16];
    tmem_ld16_sync(taddr + 16 * ch, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
    tmem_st16(taddr + 16 * ch, v);
  }
}
__device__ __forceinline__ void scale_p(uint32_t taddr, int pieces, float alpha) {
  // Two steps: alpha may be below fp16's least number, and its products with weights not.
  const bool far = alpha < 0x1p-24f;
  const __half2 by = __float2half2_rn(far ? 0x1p-15f : alpha), more = __float2half2_rn(far ? alpha * 0x1p15f : 1.f);
  const bool any_far = __any_sync(0xffffffffu, far);
#pragma unroll 1
  for (int ch = 0; ch < pieces; ++ch) {
    uint32_t v[16];
    tmem_ld16_sync(taddr + 16 * ch, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&v[e]), by);
      if (any_far) y = __hmul2(y, more);
      v[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    tmem_st16(taddr + 16 * ch, v);
  }
}

// The weights 2^(score * ks + log2 vs - ref) of a row as fp16 over its first 64 columns; `sum` gets them, each over its vs.
// Where a weight would be more than 2^(kTop + kMost), the row's reference moves by a whole number and what has been
// summed up, O (where there is one) among it, is rescaled.
template <bool kMask>
__device__ __forceinline__ void row_weights(uint32_t taddr, uint32_t orow, bool has_o, const TileInfo& info, float factor, float& ref,
                                            float& sum, int nvis) {
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    if (kMask && !__any_sync(0xffffffffu, nvis > 32 * h)) {  // (no row of the warp sees more)
      const uint32_t none[16] = {};
      tmem_st16(taddr + 16 * h, none);
      continue;
    }
    uint32_t a[32];
    tmem_ld32_issue(taddr + 32 * h, a);
    const float k0 = factor * info.ks[2 * h], k1 = factor * info.ks[2 * h + 1];
    float m0 = info.lv[2 * h] - ref, m1 = info.lv[2 * h + 1] - ref;
    tmem_ld32_wait(a);
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float ya, yb;
      ffma2(ya, yb, __uint_as_float(a[2 * q]), __uint_as_float(a[2 * q + 1]), q < 8 ? k0 : k1, q < 8 ? m0 : m1);
      if (kMask && 32 * h + 2 * q >= nvis) ya = -INFINITY;
      if (kMask && 32 * h + 2 * q + 1 >= nvis) yb = -INFINITY;
      a[2 * q] = __float_as_uint(ya);
      a[2 * q + 1] = __float_as_uint(yb);
      top[q & 3] = fmax3(top[q & 3], ya, yb);
    }
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (__any_sync(0xffffffffu, most > kTop + kMost)) {  // (rare)
      const float by = most > kTop + kMost ? ceilf(most - kTop) : 0.f, alpha = exp2f(-by);
      // (what is read again here may still be on its way: weights of the quarters before, O of a move before)
      tmem_st_wait();
      if (has_o) scale_o(orow, alpha);
      scale_p(taddr, h, alpha);
      sum *= alpha;
      ref += by;
#pragma unroll
      for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) - by);
    }
    uint32_t pw[16];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int k = 16 * b + 2 * q;
        const float pa = ex2_approx(__uint_as_float(a[k])), pb = ex2_approx(__uint_as_float(a[k + 1]));
        if (q & 1) fadd2(ls[2], ls[3], pa, pb);
        else fadd2(ls[0], ls[1], pa, pb);
        const __half2 h2 = __floats2half2_rn(pa, pb);
        pw[8 * b + q] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      sum = fmaf((ls[0] + ls[1]) + (ls[2] + ls[3]), info.iv[2 * h + b], sum);
    }
    tmem_st16(taddr + 16 * h, pw);
  }
}

__device__ void softmax_warps(const Q8Params& P, Ctl& c, uint8_t* qbuf, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3;        // TMEM lane quarter of this warp
  const int w = (warp - 2) >> 2;  // its row tile
  const int r = wq * 32 + lane;   // its row
  const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
  const uint32_t srow = tmem + lane_off + 128u * w, orow = tmem + lane_off + kOCol + 128u * w;
  volatile int* abort_flag = &c.abort_flag;
  uint32_t n = 0;           // tiles of the run so far
  uint32_t tc = 0, oc = 0;  // of this row tile: key tiles, units
  const int rj = r >> P.gp_log2, rg = r & ((1 << P.gp_log2) - 1);
  const float sign = P.scale_log2 < 0.f ? -1.f : 1.f;  // (a negative scale turns Q round)
  bool ok = true;

  float next_factor = 0.f;  // of the unit whose Q is in place: |scale| log2(e) / c
  // The warp's rows of Q times a power of two, in fp16; half a warp loads a row.  (S of the unit before has been made: Q
  // may be overwritten.)
  const auto put_q = [&](const Item& item) {
    const int64_t token0 = static_cast<int64_t>(item.t0) + item.j0 + w * (128 >> P.gp_log2);
    const int tokens = tokens_of(P, item.nq, w), chunk = lane & 15;
    uint4 raw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = wq * 32 + 2 * i + (lane >> 4), j = row >> P.gp_log2, g = row & ((1 << P.gp_log2) - 1);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (j < tokens && g < P.group)
        raw[i] = __ldg(reinterpret_cast<const uint4*>(P.q + ((token0 + j) * P.hq + static_cast<int64_t>(item.head) * P.group + g) * 128) + chunk);
    }
    // the largest size: bf16 bits without their signs compare as whole numbers, two at a time
    uint32_t both_tops = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t y[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) both_tops = __vmaxu2(both_tops, y[e] & 0x7fff7fffu);
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, max(both_tops & 0xffffu, both_tops >> 16));
    if (top >= 0x7f80u) {  // (rare) the largest finite one; what is not finite becomes NaN, and its row with it
      top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t* y = reinterpret_cast<uint32_t*>(&raw[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = y[e] & 0x7fffu, b = y[e] >> 16 & 0x7fffu;
          top = max(top, max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u));
          if (a >= 0x7f80u) y[e] |= 0x7fffu;
          if (b >= 0x7f80u) y[e] |= 0x7fff0000u;
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    // largest c in [1, 2)
    const int e = min(max(static_cast<int>(top >> 7) - 127, -126), 126);
    const float up = __int_as_float((127 - e) << 23) * sign;
    next_factor = fabsf(P.scale_log2) * (e >= -100 ? __int_as_float((127 + e) << 23) : 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = wq * 32 + 2 * i + (lane >> 4);
      const uint32_t y[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 z = __floats2half2_rn(__uint_as_float(y[k] << 16) * up, __uint_as_float(y[k] & 0xffff0000u) * up);
        h[k] = *reinterpret_cast<const uint32_t*>(&z);
      }
      *reinterpret_cast<uint4*>(qbuf + w * kTileBytes + (chunk >> 3) * kHalfBytes + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) =
          make_uint4(h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.q_full[w]);
  };

  Item item{};
  // (the first pass has no unit to work on: it only puts Q in place)
  for (uint32_t next = 0; ok; ++next) {
    const bool none = next == 0;
    const int nq = none ? 0 : tokens_of(P, item.nq, w), j0 = item.j0 + w * (128 >> P.gp_log2);
    const int slot = (next + kItemRing - 1) % kItemRing;  // of this unit
    const bool live = rj < nq && rg < P.group;  // a real (token, head) row
    const bool warp_live = __any_sync(0xffffffffu, live);
    const float factor = next_factor;
    float ref = -INFINITY, sum = 0.f;
#pragma unroll 1
    for (int j = 0; j < item.nt && nq > 0; ++j, ++n) {
      const int k0 = (item.kt0 + j) * kTileKeys;
      const int nvis = max(0, min(kTileKeys, item.ctx + j0 + rj + 1 - k0));
      const bool edge = k0 + kTileKeys > item.ctx + item.j0 + 1;             // not every row of the unit sees all of the tile
      const bool masked = edge && __any_sync(0xffffffffu, nvis < kTileKeys);  // nor of the warp
      ok = all(wait_for(&c.s_full[w], tc++ & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      // (S of this tile is complete, and with it every MMA of the row tile that was issued before)
      const TileInfo& info = c.info[n & 3];
      if (warp_live) {
        // a row's first reference; without one (it has seen nothing yet) all its weights are 0
        if (__any_sync(0xffffffffu, ref == -INFINITY)) {
          const float top = masked ? row_largest<true>(srow, info, factor, nvis) : row_largest<false>(srow, info, factor, kTileKeys);
          if (ref == -INFINITY) ref = top - kTop;
        }
        float use = ref == -INFINITY ? 0.f : ref;
        if (masked) row_weights<true>(srow, orow, j > 0, info, factor, use, sum, nvis);
        else row_weights<false>(srow, orow, j > 0, info, factor, use, sum, kTileKeys);
        if (ref != -INFINITY) ref = use;
        tmem_st_wait();
        if (edge) {
          ok = all(wait_for(&c.vfull[n % kStages], (n / kStages) & 1, abort_flag));
          uint32_t seen = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int vis = min(max(nvis - 32 * k, 0), 32);
            seen |= info.spoilt[k] & (vis == 32 ? 0xffffffffu : (1u << vis) - 1u);
          }
          if (seen) sum = __int_as_float(0x7fffffff);
        }
      }  // (otherwise no row of this warp is stored: its P may hold anything)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.p_full[w]);
      if (!ok) break;
    }
    if (!ok) break;
    // the next unit's Q first: its S is made while this unit's rows are stored
    ok = all(wait_for(&c.item_full[next % kItemRing], (next / kItemRing) & 1, abort_flag));
    if (!ok) break;
    const Item after = c.ring[next % kItemRing];
    if (after.idx >= 0 && tokens_of(P, after.nq, w) > 0) put_q(after);
    if (nq == 0) {  // no unit, or one without rows of this tile
      n += item.nt;
      __syncwarp();
      if (!none && lane == 0) mbar_arrive(&c.item_empty[slot]);
      if (after.idx < 0) break;
      item = after;
      continue;
    }
    ok = all(wait_for(&c.o_full[w], oc++ & 1, abort_flag));
    if (!ok) break;
    tc_fence_after();
    const bool bad = *reinterpret_cast<volatile int*>(&c.bad[slot]) != 0;
    const int part = item.slot, row = 128 * w + r;
    // where the row goes: the output, or its partial
    uint8_t* dst = part < 0 ? reinterpret_cast<uint8_t*>(P.out + ((static_cast<int64_t>(item.t0) + j0 + rj) * P.hq +
                                                                  static_cast<int64_t>(item.head) * P.group + rg) * 128)
                            : reinterpret_cast<uint8_t*>(P.part_o + (static_cast<int64_t>(part) * P.rows_cap + row) * 128);
    const bool zero = bad || sum == 0.f;
    const float inv = 1.f / sum;
#pragma unroll 1  // a quarter of the row at a time keeps the code and the registers small
    for (int g = 0; g < 4; ++g) {
      uint32_t v[32];
      tmem_ld32_issue(orow + 32 * g, v);
      tmem_ld32_wait(v);
      if (live && part >= 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) st_global_v8(dst + 128 * g + 32 * k, *reinterpret_cast<const uint32_t(*)[8]>(v + 8 * k));
      } else if (live) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t wv[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 h2 =
                __floats2bfloat162_rn(__uint_as_float(v[16 * k + 2 * e]) * inv, __uint_as_float(v[16 * k + 2 * e + 1]) * inv);
            wv[e] = zero ? 0u : *reinterpret_cast<const uint32_t*>(&h2);
          }
          uint8_t* to = dst + 64 * g + 32 * k;
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
    if (live && part >= 0) {
      float* ml = P.part_ml + (static_cast<int64_t>(part) * P.rows_cap + row) * 2;
      // (of a row that saw nothing, or a NaN, the sum says it all; a sum of -1: a bad block id)
      ml[0] = sum != 0.f && sum == sum ? ref : -INFINITY;
      ml[1] = bad ? -1.f : sum;
    }
    // O has been read: the next unit's first P V may overwrite it
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&c.o_free[w]);
      mbar_arrive(&c.item_empty[slot]);
    }
    if (after.idx < 0) break;
    item = after;
  }
  if (!ok && !*abort_flag && lane == 0) raise_abort(c, P.err);
}

__global__ void __launch_bounds__(kThreads, 1) q8_chunk_kernel(const Q8Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qbuf = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* kbuf = qbuf + 2 * kTileBytes;
  uint8_t* vbuf = kbuf + kStages * kTileBytes;
  Ctl& c = *reinterpret_cast<Ctl*>(vbuf + kStages * kTileBytes);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&c.kfull[s], 4);
      mbar_init(&c.kempty[s], 1);
      mbar_init(&c.vfull[s], 4);
      mbar_init(&c.vempty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&c.s_full[w], 1);
      mbar_init(&c.p_full[w], 4);
      mbar_init(&c.o_full[w], 1);
      mbar_init(&c.o_free[w], 4);
      mbar_init(&c.q_full[w], 4);
    }
    for (int s = 0; s < kItemRing; ++s) {
      mbar_init(&c.item_full[s], 1);
      mbar_init(&c.item_empty[s], 13);  // MMA warp, softmax and converting warps
    }
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  grid_dep_wait();
  grid_dep_launch();
  find_run(P, c.run);
  if (warp == 0) walk_warp(P, c);
  else if (warp == 1) mma_warp(P, c, qbuf, kbuf, vbuf, tmem);
  else if (warp < 10) softmax_warps(P, c, qbuf, tmem);
  else convert_warps(P, c, kbuf, vbuf);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int launch_q8_chunks(const Q8Params& p, int ctas, cudaStream_t s) {
  static uint64_t smem_set = 0;
  const int st = set_smem_once(reinterpret_cast<const void*>(q8_chunk_kernel), kSmemBytes, &smem_set);
  return st ? st : cuda_status(launch_k(q8_chunk_kernel, dim3(ctas), dim3(kThreads), kSmemBytes, s, p));
}

}  // namespace pkv
