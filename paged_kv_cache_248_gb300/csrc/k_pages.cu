// k_pages.cu -- the pages of a cache whose requests carry several candidate
// continuations: the accepted path of a drafted tree moved together, and block tables
// reordered after the beams they continue, with reference counts, freed and fresh blocks
// and copy-on-write on the device ("The 1960s Operating System Trick ..." page,
// Technical Details: samples share blocks until they diverge, and a block without users
// is free again).
//
// Both move bytes and count; neither computes.  They are bound by launch and memory latency at one
// layer; over the layers of a model forking is bound by HBM, moving a path still by latency.
#include "pkv_internal.cuh"

namespace pkv {
namespace {

// ------------------------------------------------------------------ accepted path
// One CTA per (request, layer).  Every thread owns 16-byte columns of the request's K or
// V rows (one kv head, one piece of a row) and moves them node by node: path[a] >= a
// because the path ascends, so position c + a is never a source of a later move and a
// thread may overwrite it once it has loaded the sources up to a.  Columns are
// independent, so the threads need no order among them.  8 rows at a time hide part of the loads'
// latency, which is the bound: before its first row a CTA loads lengths, path and table, each by the
// one before.  33 requests in one layer take 2.7 us, 64 in 32 layers (12 of 64 nodes, 92 MB of reads
// and writes, 13.6 us at a copy's rate) 19.2 us, and 14.5 where L2 holds the rows; DRAM is 31 % busy.
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;     // rows a thread holds in registers between loads and stores
constexpr int kMoveChunk = 256;   // path entries staged in shared memory at a time

struct MoveParams {
  const int32_t* path;
  const int32_t* path_lens;
  const int32_t* bt;
  const int32_t* seq_lens;
  const int32_t* qsl;
  uint4* kc;
  uint4* vc;
  int32_t* new_lens;
  uint32_t* err;
  int64_t num_blocks;
  int64_t vec_per_layer;
  int32_t max_path, max_blocks, hkv, vec_per_row;
};

__global__ void __launch_bounds__(kMoveThreads) compact_path_kernel(const MoveParams P) {
  __shared__ int64_t s_src[kMoveChunk], s_dst[kMoveChunk];  // row offsets (vectors), -1: nothing to move
  grid_dep_wait();
  grid_dep_launch();
  const int i = blockIdx.x;
  const bool report = blockIdx.y == 0;
  const int64_t q_len = static_cast<int64_t>(__ldg(P.qsl + i + 1)) - __ldg(P.qsl + i);
  const int64_t L = __ldg(P.seq_lens + i);
  const int n = __ldg(P.path_lens + i);
  const int32_t* path = P.path + static_cast<int64_t>(i) * P.max_path;
  const int32_t* btrow = P.bt + static_cast<int64_t>(i) * P.max_blocks;
  const int64_t c0 = L - q_len;
  uint32_t bad = 0;
  if (q_len < 0 || c0 < 0 || (L + kBlock - 1) / kBlock > P.max_blocks || n < 0 || n > P.max_path || n > q_len)
    bad = kErrLength;
  if (!bad) {  // the whole path, before anything moves
    for (int a = threadIdx.x; a < n; a += kMoveThreads) {
      const int u = __ldg(path + a);
      const int prev = a ? __ldg(path + a - 1) : -1;
      if (u <= prev || u >= q_len) {
        bad |= kErrLength;
      } else {
        const int32_t bs = __ldg(btrow + (c0 + u) / kBlock), bd = __ldg(btrow + (c0 + a) / kBlock);
        if (bs < 0 || bs >= P.num_blocks || bd < 0 || bd >= P.num_blocks) bad |= kErrBlockId;
      }
    }
  }
  const int any_len = __syncthreads_or(bad & kErrLength);
  const int any_block = __syncthreads_or(bad & kErrBlockId);
  if (any_len || any_block) {
    if (report && threadIdx.x == 0) {
      flag_error(P.err, (any_len ? kErrLength : 0u) | (any_block ? kErrBlockId : 0u));
      P.new_lens[i] = static_cast<int32_t>(L);
    }
    return;
  }
  if (report && threadIdx.x == 0) P.new_lens[i] = static_cast<int32_t>(c0 + n);
  const int64_t row_vecs = P.vec_per_row, block_vecs = static_cast<int64_t>(P.hkv) * kBlock * row_vecs;
  const int cols = 2 * P.hkv * P.vec_per_row;
  for (int a0 = 0; a0 < n; a0 += kMoveChunk) {
    const int m = min(kMoveChunk, n - a0);
    __syncthreads();
    for (int a = threadIdx.x; a < m; a += kMoveThreads) {
      const int u = __ldg(path + a0 + a);
      const int64_t ps = c0 + u, pd = c0 + a0 + a;
      s_src[a] = u == a0 + a ? -1 : __ldg(btrow + ps / kBlock) * block_vecs + (ps % kBlock) * row_vecs;
      s_dst[a] = __ldg(btrow + pd / kBlock) * block_vecs + (pd % kBlock) * row_vecs;
    }
    __syncthreads();
    for (int col = threadIdx.x; col < cols; col += kMoveThreads) {
      const int half = col / (P.hkv * P.vec_per_row);  // 0: K, 1: V
      const int c = col - half * P.hkv * P.vec_per_row;
      const int h = c / P.vec_per_row, v = c - h * P.vec_per_row;
      uint4* base = (half ? P.vc : P.kc) + blockIdx.y * P.vec_per_layer + h * (kBlock * row_vecs) + v;
      for (int a = 0; a < m; a += kMoveBatch) {
        uint4 w[kMoveBatch];
#pragma unroll
        for (int k = 0; k < kMoveBatch; ++k)
          if (a + k < m && s_src[a + k] >= 0) w[k] = base[s_src[a + k]];
#pragma unroll
        for (int k = 0; k < kMoveBatch; ++k)
          if (a + k < m && s_src[a + k] >= 0) base[s_dst[a + k]] = w[k];
      }
    }
  }
}

// ------------------------------------------------------------------ forked tables
// Three launches, or two for few rows.  fork_gather_kernel (a CTA per row): the new row's kept blocks, and the
// old row's part of the reference counts -- an entry that k new rows keep changes by
// k - 1, in one atomic (integer sums, so their order does not matter).  fork_assign_kernel
// (one CTA): which rows copy their last block, how many fresh blocks each row needs, and
// the free blocks in order of their ids, found by a scan of the counts that stops as soon
// as every row has its blocks (130000 counts, if the free ones come last, take 30 us).  fork_finish_kernel (a CTA per row, layer and slice): the
// copies and the counts of copied and fresh blocks; after an error, everything back.
// 64 requests of 8 beams and 16 layers copy 503 MB: 74 us, a copy's rate (the first two launches hide
// behind the copies of the call before).  One request of 5 beams takes 6.3 to 7.2 us, all of it latency.
//
// Up to 32 rows of up to kFewBlocks blocks: the assigning CTA gathers by itself, a warp per row,
// which saves a launch: 0.5 us less for 5 rows of 20 blocks and for 32 of 32, as long for 32 of 128,
// 3 us more for 32 of 512; and 2 us less on the host.
constexpr int kForkThreads = 256;
constexpr int kAssignThreads = 1024;
constexpr int kForkMaxRows = 4096;
constexpr int kRowsPerThread = kForkMaxRows / kAssignThreads;
constexpr int kFewRows = kAssignThreads / 32;
constexpr int kFewBlocks = 128;

struct ForkParams {
  const int32_t* bt;
  const int32_t* lens;
  const int32_t* parents;
  int32_t* refs;
  int32_t* new_bt;
  int32_t* new_lens;
  uint4* kc;
  uint4* vc;
  uint32_t* err;
  int32_t* row_state;  // [rows] gather: 0 done, 1 done and bad entry or length, 2 bad parent (no counts touched)
  int32_t* copy_src;   // [rows] the block a row copies, -1: none
  int32_t* copy_dst;   // [rows]
  int32_t* verdict;    // [1] 0: go on, 1: undo the counts, 2: nothing to undo
  int64_t num_blocks;
  int64_t vec_per_block;
  int64_t vec_per_layer;
  int32_t rows, max_blocks, num_new, layers, slices;
};

__device__ __forceinline__ int held_blocks(int n) { return n / kBlock + (n % kBlock != 0 ? 1 : 0); }  // (n >= 0)

// How many rows continue row b (all threads of the CTA call; the result is for all), and
// whether some parent is out of range.
__device__ int count_children(const ForkParams& P, int b, int* invalid) {
  int mine = 0, bad = 0;
  for (int r = threadIdx.x; r < P.rows; r += blockDim.x) {
    const int p = __ldg(P.parents + r);
    mine += p == b ? 1 : 0;
    bad |= p < -1 || p >= P.rows ? 1 : 0;
  }
  __shared__ int s_sum[32];
  *invalid = __syncthreads_or(bad);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = mine;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) total += s_sum[w];
  __syncthreads();
  return total;
}

// The counts that old row b changes: `sign` 1 applies them, -1 takes them back.  Returns
// whether an entry is out of range.
__device__ __forceinline__ int apply_counts(const ForkParams& P, int b, int held, int children, int sign, int first, int step) {
  const int32_t* row = P.bt + static_cast<int64_t>(b) * P.max_blocks;
  int bad = 0;
  for (int m = first; m < P.max_blocks; m += step) {
    const int32_t x = __ldg(row + m);
    if (x >= P.num_blocks || (x < 0 && m < held)) {
      bad = 1;
    } else if (x >= 0) {
      const int delta = (m < held ? children : 0) - 1;
      if (delta != 0) atomicAdd(P.refs + x, sign * delta);
    }
  }
  return bad;
}

// Row b of the new tables, and the counts that old row b changes: the part of thread `first`
// of `step`, of which one reports.  Returns whether an entry is out of range.
__device__ __forceinline__ int gather_row(const ForkParams& P, int b, int children, int first, int step, bool* wrong_length) {
  const int len = __ldg(P.lens + b);
  const int p = __ldg(P.parents + b);
  int n = p >= 0 ? __ldg(P.lens + p) : 0;
  const bool len_ok = len >= 0 && held_blocks(len) <= P.max_blocks;
  const int bad = apply_counts(P, b, len_ok ? held_blocks(len) : 0, children, 1, first, step);
  n = n < 0 || held_blocks(n) > P.max_blocks ? 0 : n;
  const int held = held_blocks(n);
  // the new row must hold its fresh blocks too
  const bool fits = p < 0 || (static_cast<int64_t>(n) + P.num_new + kBlock - 1) / kBlock <= P.max_blocks;
  for (int m = first; m < P.max_blocks; m += step)
    P.new_bt[static_cast<int64_t>(b) * P.max_blocks + m] =
        m < held ? __ldg(P.bt + static_cast<int64_t>(p) * P.max_blocks + m) : -1;
  if (first == 0) P.new_lens[b] = n;
  *wrong_length = !len_ok || !fits;
  return bad;
}

__device__ __forceinline__ void report_row(const ForkParams& P, int b, bool bad, bool wrong_length) {
  P.row_state[b] = bad || wrong_length ? 1 : 0;
  if (bad) flag_error(P.err, kErrBlockId);
  if (wrong_length) flag_error(P.err, kErrLength);
}

__global__ void __launch_bounds__(kForkThreads) fork_gather_kernel(const ForkParams P) {
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x;
  int invalid = 0;
  const int children = count_children(P, b, &invalid);
  if (invalid) {
    if (threadIdx.x == 0) {
      P.row_state[b] = 2;
      if (b == 0) flag_error(P.err, kErrLength);
    }
    return;
  }
  bool wrong_length;
  const int bad = gather_row(P, b, children, threadIdx.x, kForkThreads, &wrong_length);
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) report_row(P, b, any, wrong_length);
}

// Exclusive prefix of one value per thread over the CTA; *total is the sum.
__device__ int block_exclusive(int x, int* total) {
  __shared__ int s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  __syncthreads();  // the previous use of s_warp is over
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int w = s_warp[lane], wi = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, wi, d);
    if (lane >= d) wi += y;
  }
  *total = __shfl_sync(0xffffffffu, wi, 31);
  return incl - x + __shfl_sync(0xffffffffu, wi - w, warp);
}

template <bool kFew>
__global__ void __launch_bounds__(kAssignThreads, 1) fork_assign_kernel(const ForkParams P) {
  extern __shared__ int32_t sm[];
  // a hash table of the shared last blocks (id, rows that end in it, the lowest of them)
  // and the running number of fresh blocks per row
  int slots = 32;
  while (slots < 2 * P.rows) slots *= 2;
  int32_t* h_key = sm;
  int32_t* h_cnt = sm + slots;
  int32_t* h_min = sm + 2 * slots;
  int32_t* start = sm + 3 * slots;  // [rows + 1]
  int32_t* info = start + P.rows + 1;  // [rows] held blocks * 2 + copies
  for (int s = threadIdx.x; s < slots; s += kAssignThreads) {
    h_key[s] = -1;
    h_cnt[s] = 0;
    h_min[s] = 0x7fffffff;
  }
  grid_dep_wait();
  grid_dep_launch();
  int state = 0;
  if (kFew) {  // gather, a warp per row
    const int b = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int p = lane < P.rows ? __ldg(P.parents + lane) : -1;
    const bool invalid = __any_sync(0xffffffffu, p < -1 || p >= P.rows);
    const int children = __popc(__ballot_sync(0xffffffffu, p == b));
    if (invalid) {
      if (threadIdx.x == 0) {
        P.row_state[0] = 2;
        flag_error(P.err, kErrLength);
      }
    } else if (b < P.rows) {
      bool wrong_length;
      const int bad = gather_row(P, b, children, lane, 32, &wrong_length);
      const bool any = __any_sync(0xffffffffu, bad != 0);
      if (lane == 0) report_row(P, b, any, wrong_length);
    }
    __syncthreads();
  }
  for (int r = threadIdx.x; r < P.rows; r += kAssignThreads) state |= __ldcg(P.row_state + r);
  state = __syncthreads_or(state & 2) ? 2 : (__syncthreads_or(state & 1) ? 1 : 0);
  if (state) {
    if (threadIdx.x == 0) *P.verdict = state;
    return;
  }
  // row b is thread b's mod 1024; the loads of all its rows come before the table's loops, whose
  // threads part ways
  int last[kRowsPerThread], place[kRowsPerThread], held[kRowsPerThread], grow[kRowsPerThread];
#pragma unroll
  for (int k = 0; k < kRowsPerThread; ++k) {
    const int b = threadIdx.x + k * kAssignThreads;
    last[k] = -1;
    held[k] = grow[k] = place[k] = 0;
    if (b < P.rows) {
      const int n = __ldcg(P.new_lens + b);
      const int p = __ldg(P.parents + b);
      held[k] = held_blocks(n);
      grow[k] = p >= 0 ? static_cast<int>((static_cast<int64_t>(n) + P.num_new + kBlock - 1) / kBlock) - held[k] : 0;
      if (n % kBlock != 0 && P.num_new > 0)
        last[k] = __ldcg(P.new_bt + static_cast<int64_t>(b) * P.max_blocks + held[k] - 1);
    }
  }
  int users[kRowsPerThread];
#pragma unroll
  for (int k = 0; k < kRowsPerThread; ++k) users[k] = last[k] >= 0 ? __ldcg(P.refs + last[k]) : 0;
#pragma unroll
  for (int k = 0; k < kRowsPerThread; ++k) {
    if (k * kAssignThreads >= P.rows) break;
    if (last[k] >= 0) {
      uint32_t s = (static_cast<uint32_t>(last[k]) * 2654435761u) & (slots - 1);
      while (true) {  // at most `rows` keys in at least 2 * rows slots
        const int32_t old = atomicCAS(&h_key[s], -1, last[k]);
        if (old == -1 || old == last[k]) break;
        s = (s + 1) & (slots - 1);
      }
      place[k] = static_cast<int>(s);
      atomicAdd(&h_cnt[s], 1);
      atomicMin(&h_min[s], static_cast<int>(threadIdx.x) + k * kAssignThreads);
    }
    __syncwarp();
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int k = 0; k < kRowsPerThread; ++k) {
    if (k * kAssignThreads >= P.rows) break;
    const int b = threadIdx.x + k * kAssignThreads;
    const bool copy = last[k] >= 0 && (users[k] > h_cnt[place[k]] || h_min[place[k]] != b);
    int sum = 0;
    const int at = total + block_exclusive((copy ? 1 : 0) + grow[k], &sum);
    if (b < P.rows) {
      info[b] = held[k] * 2 + (copy ? 1 : 0);
      P.copy_src[b] = copy ? last[k] : -1;
      start[b] = at;
    }
    total += sum;
  }
  if (threadIdx.x == 0) start[P.rows] = total;
  __syncthreads();
  // free blocks in order of their ids
  int found = 0;
  for (int64_t x0 = 0; x0 < P.num_blocks && found < total; x0 += kAssignThreads * 4) {
    const int64_t x = x0 + threadIdx.x * 4;
    int free_bits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x + e < P.num_blocks && __ldcg(P.refs + x + e) == 0) free_bits |= 1 << e;
    int here = 0;
    int rank = found + block_exclusive(__popc(free_bits), &here);
    while (free_bits && rank < total) {
      const int e = __ffs(free_bits) - 1;
      free_bits &= free_bits - 1;
      int lo = 0, hi = P.rows - 1;  // the last row that starts at or before this rank
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= rank) lo = mid; else hi = mid - 1;
      }
      const int off = rank - start[lo], copy = info[lo] & 1, h = info[lo] >> 1;
      const int32_t id = static_cast<int32_t>(x + e);
      if (copy && off == 0) {
        P.copy_dst[lo] = id;
        P.new_bt[static_cast<int64_t>(lo) * P.max_blocks + h - 1] = id;
      } else {
        P.new_bt[static_cast<int64_t>(lo) * P.max_blocks + h + off - copy] = id;
      }
      ++rank;
    }
    found += here;
  }
  if (threadIdx.x == 0) {
    *P.verdict = found < total ? 1 : 0;
    if (found < total) flag_error(P.err, kErrNoPages);
  }
}

__global__ void __launch_bounds__(kForkThreads) fork_finish_kernel(const ForkParams P) {
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x;
  const int layer = blockIdx.y / P.slices, slice = blockIdx.y % P.slices;
  const int verdict = __ldcg(P.verdict);
  if (verdict != 0) {  // everything as it was
    if (blockIdx.y != 0) return;
    if (verdict == 1) {
      int invalid = 0;
      const int children = count_children(P, b, &invalid);
      const int len = __ldg(P.lens + b);
      apply_counts(P, b, len >= 0 && held_blocks(len) <= P.max_blocks ? held_blocks(len) : 0, children, -1, threadIdx.x, kForkThreads);
    }
    for (int m = threadIdx.x; m < P.max_blocks; m += kForkThreads)
      P.new_bt[static_cast<int64_t>(b) * P.max_blocks + m] = __ldg(P.bt + static_cast<int64_t>(b) * P.max_blocks + m);
    if (threadIdx.x == 0) P.new_lens[b] = __ldg(P.lens + b);
    return;
  }
  const int32_t src = __ldcg(P.copy_src + b);
  if (blockIdx.y == 0) {  // the counts of this row's copied and fresh blocks
    const int n = __ldcg(P.new_lens + b);
    const int held = held_blocks(n);
    const int most = __ldg(P.parents + b) >= 0 ? static_cast<int>((static_cast<int64_t>(n) + P.num_new + kBlock - 1) / kBlock) : 0;
    for (int m = held + threadIdx.x; m < most; m += kForkThreads)
      P.refs[__ldcg(P.new_bt + static_cast<int64_t>(b) * P.max_blocks + m)] = 1;
    if (threadIdx.x == 0 && src >= 0) {
      atomicAdd(P.refs + src, -1);
      P.refs[__ldcg(P.copy_dst + b)] = 1;
    }
  }
  if (src < 0 || P.kc == nullptr) return;
  const int32_t dst = __ldcg(P.copy_dst + b);
  const int64_t per_slice = (P.vec_per_block + P.slices - 1) / P.slices;
  const int64_t begin = slice * per_slice;
  const int64_t end = begin + per_slice < P.vec_per_block ? begin + per_slice : P.vec_per_block;
  uint4* k = P.kc + layer * P.vec_per_layer;
  uint4* v = P.vc + layer * P.vec_per_layer;
  constexpr int kUnroll = 4;
  for (int64_t c0 = begin + threadIdx.x; c0 < end; c0 += kForkThreads * kUnroll) {
    uint4 a[kUnroll], d[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + static_cast<int64_t>(u) * kForkThreads;
      if (c < end) {
        a[u] = k[src * P.vec_per_block + c];
        d[u] = v[src * P.vec_per_block + c];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + static_cast<int64_t>(u) * kForkThreads;
      if (c < end) {
        k[dst * P.vec_per_block + c] = a[u];
        v[dst * P.vec_per_block + c] = d[u];
      }
    }
  }
}

size_t assign_smem(int rows) {
  int slots = 32;
  while (slots < 2 * rows) slots *= 2;
  return (3 * static_cast<size_t>(slots) + 2 * static_cast<size_t>(rows) + 1) * sizeof(int32_t);
}

int64_t elem_bytes(const pkv_cache_desc& c) { return c.dtype == PKV_F32 ? 4 : 2; }

}  // namespace

int launch_compact_path(const int32_t* path, int32_t max_path, const int32_t* path_lens, const int32_t* bt,
                        int32_t max_blocks, const int32_t* seq_lens, const int32_t* qsl, int32_t num_seqs, void* kc,
                        void* vc, const pkv_cache_desc& c, int32_t num_layers, int32_t* new_lens, uint32_t* err,
                        cudaStream_t s) {
  MoveParams p{};
  p.path = path;
  p.path_lens = path_lens;
  p.bt = bt;
  p.seq_lens = seq_lens;
  p.qsl = qsl;
  p.kc = static_cast<uint4*>(kc);
  p.vc = static_cast<uint4*>(vc);
  p.new_lens = new_lens;
  p.err = err;
  p.num_blocks = c.num_blocks;
  p.max_path = max_path;
  p.max_blocks = max_blocks;
  p.hkv = c.num_kv_heads;
  p.vec_per_row = static_cast<int32_t>(c.head_dim * elem_bytes(c) / 16);
  p.vec_per_layer = c.num_blocks * c.num_kv_heads * kBlock * p.vec_per_row;
  return cuda_status(launch_k(compact_path_kernel, dim3(num_seqs, num_layers), dim3(kMoveThreads), 0, s, p));
}

size_t fork_workspace(int32_t num_rows) {
  return ((3 * static_cast<size_t>(num_rows) + 1) * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
}

int launch_fork_tables(const int32_t* bt, const int32_t* lens, int32_t rows, int32_t max_blocks, const int32_t* parents,
                       int32_t num_new, int32_t* refs, int32_t* new_bt, int32_t* new_lens, void* kc, void* vc,
                       const pkv_cache_desc& c, int32_t num_layers, void* workspace, int num_sms, uint32_t* err,
                       cudaStream_t s) {
  ForkParams p{};
  p.bt = bt;
  p.lens = lens;
  p.parents = parents;
  p.refs = refs;
  p.new_bt = new_bt;
  p.new_lens = new_lens;
  p.kc = static_cast<uint4*>(kc);
  p.vc = static_cast<uint4*>(vc);
  p.err = err;
  p.verdict = static_cast<int32_t*>(workspace);
  p.row_state = p.verdict + 1;
  p.copy_src = p.row_state + rows;
  p.copy_dst = p.copy_src + rows;
  p.num_blocks = c.num_blocks;
  p.vec_per_block = c.num_kv_heads * kBlock * c.head_dim * elem_bytes(c) / 16;
  p.vec_per_layer = c.num_blocks * p.vec_per_block;
  p.rows = rows;
  p.max_blocks = max_blocks;
  p.num_new = num_new;
  p.layers = kc ? num_layers : 1;
  p.slices = 1;
  while (kc && static_cast<int64_t>(rows) * p.layers * p.slices < 2LL * num_sms && p.vec_per_block / (p.slices * 2) >= kForkThreads)
    p.slices *= 2;
  const size_t smem = assign_smem(rows);
  int st;
  if (rows <= kFewRows && max_blocks <= kFewBlocks) {
    st = cuda_status(launch_k(fork_assign_kernel<true>, dim3(1), dim3(kAssignThreads), smem, s, p));
  } else {
    static uint64_t smem_set = 0;
    st = set_smem_once(reinterpret_cast<const void*>(fork_assign_kernel<false>),
                       static_cast<int>(assign_smem(kForkMaxRows)), &smem_set);
    if (st) return st;
    st = cuda_status(launch_k(fork_gather_kernel, dim3(rows), dim3(kForkThreads), 0, s, p));
    if (st) return st;
    st = cuda_status(launch_k(fork_assign_kernel<false>, dim3(1), dim3(kAssignThreads), smem, s, p));
  }
  if (st) return st;
  return cuda_status(launch_k(fork_finish_kernel, dim3(rows, p.layers * p.slices), dim3(kForkThreads), 0, s, p));
}

}  // namespace pkv
