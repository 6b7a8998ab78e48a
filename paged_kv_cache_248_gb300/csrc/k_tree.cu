// k_tree.cu -- attention of drafted tokens, which form a tree, over an fp32 paged cache, on
// CUDA cores; and the ancestor masks of such trees.
//
// Mathematics.  Node j of request i sees the keys u < c_i = seq_len - q_len, and of the
// draft the keys c_i + b whose bit b its mask row has; out = sum_u softmax_u(scale q.K_u) V_u
// over those keys alone, with the softmax's running maximum and sum in fp32.  Keys that are
// not seen are never multiplied with anything, so whatever they hold stays out.
#include "pkv_internal.cuh"
#include "ptx.cuh"
#include "tree_merge.cuh"

namespace pkv {
namespace {

// ------------------------------------------------------------------ ancestor masks
// A thread per node follows its parents to the context and sets their bits in its own
// mask row.  Parents have smaller indices, so the walk ends after at most q_len steps.
__global__ void __launch_bounds__(128) tree_mask_kernel(const int32_t* __restrict__ parents,
                                                        const int32_t* __restrict__ qsl, int num_seqs,
                                                        int64_t num_tokens, uint64_t* __restrict__ mask, int words,
                                                        int32_t* __restrict__ depths, uint32_t* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= num_tokens) return;
  const int i = find_seq(qsl, num_seqs, t);
  const int64_t q0 = __ldg(qsl + i), q1 = __ldg(qsl + i + 1);
  uint64_t* row = mask + t * words;
  for (int w = 0; w < words; ++w) row[w] = 0;
  int depth = 0;
  bool ok = t >= q0 && t < q1 && q1 <= num_tokens && q0 >= 0 && t - q0 < 64LL * words;
  if (ok) {
    int64_t u = t - q0;
    int64_t word = u / 64;  // ancestors come in descending order: a word is done when left
    uint64_t bits = 0;
    while (true) {
      if (u / 64 != word) {
        row[word] = bits;
        word = u / 64;
        bits = 0;
      }
      bits |= uint64_t(1) << (u % 64);
      const int p = __ldg(parents + q0 + u);
      if (p < -1 || p >= u) {
        ok = false;
        break;
      }
      if (p < 0) break;
      u = p;
      ++depth;
    }
    row[word] = bits;
  }
  if (!ok) {
    flag_error(err, kErrLength);
    for (int w = 0; w < words; ++w) row[w] = 0;
    depth = 0;
  }
  if (depths) depths[t] = depth;
}

// ------------------------------------------------------------------ CUDA-core attention
// The G query heads of a kv head and the nodes of a request are rows (node * G + head), 32 to a
// unit; a unit goes over the request's key tiles of 64 keys, K and V of which are staged in
// shared memory once for all its rows.  A thread owns 4 rows with 4 keys of the scores, and the
// same 4 rows with D / 16 columns of the result, so that the 16 threads of a row keep its
// maximum, sum and result in registers from tile to tile.  All units' key tiles, one after the
// other, are cut into equal runs, one per CTA; a unit that is cut leaves partials (accumulator,
// maximum, sum) that the merge kernel joins in the order of the keys.
//
// Bound: latency for few requests, fp32 FMAs and the shared-memory loads that feed them for many.
// 5 requests of 100 to 700 keys with 3 to 13 nodes, 8 / 2 heads of 64: 12.7 us, of which the
// joining kernel is 3 (one CTA per node and kv head, keys in turn, took 132).
// 4 requests of 4000 keys with 24 nodes, 32 / 8 heads of 64 (3.1 GFLOP): 105 us, 40 % of the FMA
// rate, with four CTAs an SM (two: 121); heads of 128 leave room for two.
constexpr int kRows = 32;      // rows of a unit
constexpr int kKeys = 64;      // keys of a tile
constexpr int kThreads = 128;
template <int D>
constexpr int kCtasPerSm = D == 64 ? 4 : 2;
constexpr float kLog2e = 1.4426950408889634f;

struct Params32 {
  TreeArgs a;
  uint32_t* err;
  float* part_o;   // [2 * runs][kRows][D]
  float* part_ml;  // [2 * runs][kRows][2]
  Cut* cuts;       // [2 * runs]
  int32_t hkv, group;
  float scale_log2;
};

struct Request32 {
  int32_t t0, q_len, len, tiles, units, cost;
  bool wrong;
};

__device__ __forceinline__ Request32 request_of(const Params32& P, int i) {
  const AttnArgs& A = P.a.a;
  Request32 r;
  const int32_t q0 = __ldg(A.qsl + i), q1 = __ldg(A.qsl + i + 1), len = __ldg(A.seq_lens + i);
  const int64_t n = static_cast<int64_t>(q1) - q0;
  const bool real = n >= 0 && q0 >= 0 && q1 <= A.num_tokens, rows = real && n > 0;
  bool fits = rows && len >= n && len <= kMaxLen && n <= A.max_query_len &&
              (static_cast<int64_t>(len) + kBlock - 1) / kBlock <= A.max_blocks;
  // (of rows that are not real, those that exist)
  r.t0 = max(q0, 0);
  r.q_len = static_cast<int32_t>(max(int64_t(0), min(static_cast<int64_t>(q1), A.num_tokens) - r.t0));
  r.len = len;
  r.tiles = static_cast<int>(static_cast<uint32_t>(len - 1) / kKeys) + 1;
  const int64_t units = (static_cast<int64_t>(r.q_len) * P.group + kRows - 1) / kRows;
  const int64_t cost = units * P.hkv * r.tiles;
  fits = fits && cost < (int64_t(1) << 31);  // (more would be terabytes of K and V, read once a unit)
  r.units = static_cast<int32_t>(units);
  r.cost = fits ? static_cast<int32_t>(cost) : 0;
  r.wrong = !real || (rows && !fits);
  return r;
}

// d += a * b, two values at a time: half the instructions of single ones, which leaves issue slots
// for the shared-memory loads.
__device__ __forceinline__ void fma_pair(float2& d, const float2& a, const float2& b) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(d.x), "+f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

// One tile's rows (K or V) into shared memory, rows past the context as zeros.
template <int D>
__device__ __forceinline__ void stage_tile(float* dst, const float* src, const int32_t* ids, int k0, int len, int head, int hkv) {
  constexpr int kVecs = D / 4;
  for (int v = threadIdx.x; v < kKeys * kVecs; v += kThreads) {
    const int key = v / kVecs, c = v % kVecs;
    float* to = dst + key * (D + 4) + 4 * c;
    if (k0 + key < len) {
      const float* from = src + ((static_cast<int64_t>(ids[key / kBlock]) * hkv + head) * kBlock + key % kBlock) * D + 4 * c;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    } else {
      *reinterpret_cast<float4*>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  cp_async_commit();
}

// The result's 4 rows += P V over a tile; kDrafted: keys of weight 0 are left out, whatever V holds.
template <int D, bool kDrafted>
__device__ __forceinline__ void add_pv(float2 (&o)[4][D / 32], const float* sp, const float* sv, int rg, int cg) {
  constexpr int C = D / 32;  // pairs of result columns
#pragma unroll 2
  for (int u = 0; u < kKeys; u += 4) {
    float4 p[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4*>(sp + (4 * rg + r) * (kKeys + 4) + u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float2 v[C];
#pragma unroll
      for (int c = 0; c < C; c += 2) {
        const float4 x = *reinterpret_cast<const float4*>(sv + (u + e) * (D + 4) + 64 * (c / 2) + 4 * cg);
        v[c] = make_float2(x.x, x.y);
        v[c + 1] = make_float2(x.z, x.w);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w = e == 0 ? p[r].x : e == 1 ? p[r].y : e == 2 ? p[r].z : p[r].w;
        if (!kDrafted || !(w == 0.f)) {
#pragma unroll
          for (int c = 0; c < C; ++c) fma_pair(o[r][c], make_float2(w, w), v[c]);
        }
      }
    }
  }
}

template <int D>
constexpr int kSmem32 = (kRows * (D + 4) + 2 * kKeys * (D + 4) + kRows * (kKeys + 4)) * static_cast<int>(sizeof(float));

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D>) tree_f32_kernel(const Params32 P) {
  constexpr int C = D / 32;  // pairs of result columns of a thread
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;
  float* sk = sq + kRows * (D + 4);
  float* sv = sk + kKeys * (D + 4);
  float* sp = sv + kKeys * (D + 4);
  __shared__ int64_t s_sum[kThreads / 32], s_base;
  __shared__ int32_t s_seq, s_ids[2][kKeys / kBlock], s_bad;
  const AttnArgs& A = P.a.a;
  const float* q = static_cast<const float*>(A.q);
  const float* kc = static_cast<const float*>(A.k_cache);
  const float* vc = static_cast<const float*>(A.v_cache);
  float* out = static_cast<float*>(A.out);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid & 15, rg = tid >> 4;
  grid_dep_wait();
  grid_dep_launch();
  // this CTA's run of key tiles
  const int per = (A.num_seqs + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, A.num_seqs), i1 = min(i0 + per, A.num_seqs);
  int64_t mine = 0;
  bool wrong = false;
  for (int i = i0; i < i1; ++i) {
    const Request32 r = request_of(P, i);
    mine += r.cost;
    wrong |= r.wrong;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (tid == 0) s_seq = 0;
  const bool any_wrong = __syncthreads_or(wrong);
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  const int64_t run = (total + gridDim.x - 1) / gridDim.x;
  int64_t pos = run * blockIdx.x;
  const int64_t end = min(total, pos + run);
  if (pos >= before && pos < before + mine) {
    int64_t at = before;
    for (int i = i0; i < i1; ++i) {
      const int cost = request_of(P, i).cost;
      if (pos < at + cost) {
        s_seq = i;
        s_base = at;
        break;
      }
      at += cost;
    }
  }
  if (any_wrong) {  // lengths that do not fit, rows that do not exist: reported, and zero as far as they do
    for (int i = blockIdx.x; i < A.num_seqs; i += gridDim.x) {
      const Request32 r = request_of(P, i);
      if (!r.wrong) continue;
      if (tid == 0) flag_error(P.err, kErrLength);
      const int64_t n = static_cast<int64_t>(r.q_len) * A.num_q_heads * D;
      for (int64_t e = tid; e < n; e += kThreads) out[static_cast<int64_t>(r.t0) * A.num_q_heads * D + e] = 0.f;
    }
  }
  if (tid < 2) P.cuts[2 * blockIdx.x + tid].parts = 0;
  __syncthreads();
  int seq = s_seq;
  int64_t base = pos < end ? s_base : 0;
  while (pos < end) {
    const Request32 rq = request_of(P, seq);
    if (pos >= base + rq.cost) {
      base += rq.cost;
      if (++seq >= A.num_seqs) break;  // (lengths that changed meanwhile)
      continue;
    }
    const uint32_t off = static_cast<uint32_t>(pos - base);
    const int unit = static_cast<int>(off / rq.tiles), first = static_cast<int>(off - unit * rq.tiles);
    const int nt = static_cast<int>(min(static_cast<int64_t>(rq.tiles - first), end - pos));
    pos += nt;
    const int head = unit / rq.units, row0 = (unit - head * rq.units) * kRows;
    const int rows = min(kRows, rq.q_len * P.group - row0), ctx = rq.len - rq.q_len;
    const int slot = nt == rq.tiles ? -1 : 2 * static_cast<int>(blockIdx.x) + (first == 0 ? 1 : 0);
    if (slot >= 0 && tid == 0) {  // the runs before that have a part of the unit, and after
      const int len = static_cast<int>(min(run, int64_t(0x3fffffff)));
      const int before = (first + len - 1) / len, after = (rq.tiles - first - nt + len - 1) / len;
      P.cuts[slot] = Cut{before + 1 + after, before, rq.t0, head, {row0, 0}, {rows, 0}};
    }
    const int32_t* btrow = A.block_tables + static_cast<int64_t>(seq) * A.max_blocks;
    // ids of the first tile; Q rows
    auto load_ids = [&](int tile, int slot2) {
      if (tid < kKeys / kBlock) {
        const int blk = tile * (kKeys / kBlock) + tid;
        int id = 0;
        if (blk * kBlock < rq.len) {
          id = __ldg(btrow + blk);
          if (id < 0 || id >= A.cache.num_blocks) {
            flag_error(P.err, kErrBlockId);
            s_bad = 1;
            id = 0;
          }
        }
        s_ids[slot2][tid] = id;
      }
    };
    if (tid == 0) s_bad = 0;
    __syncthreads();
    load_ids(first, 0);
    for (int v = tid; v < kRows * D / 4; v += kThreads) {
      const int r = v / (D / 4), c = v % (D / 4), row = row0 + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        x = __ldg(reinterpret_cast<const float4*>(
                      q + ((static_cast<int64_t>(rq.t0) + row / P.group) * A.num_q_heads + head * P.group + row % P.group) * D) + c);
      *reinterpret_cast<float4*>(sq + r * (D + 4) + 4 * c) = x;
    }
    __syncthreads();
    stage_tile<D>(sk, kc, s_ids[0], first * kKeys, rq.len, head, P.hkv);
    stage_tile<D>(sv, vc, s_ids[0], first * kKeys, rq.len, head, P.hkv);
    float m[4], l[4];
    float2 o[4][C];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) o[r][c] = make_float2(0.f, 0.f);
    }
    for (int j = 0; j < nt; ++j) {
      const int k0 = (first + j) * kKeys;
      const bool drafted = k0 + kKeys > ctx;
      if (j + 1 < nt) load_ids(first + j + 1, (j + 1) & 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");  // K has landed
      __syncthreads();
      // scores of 4 rows and keys cg, cg + 16, cg + 32, cg + 48
      // (sums of the even and of the odd columns)
      float2 s2[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) s2[r][e] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4*>(sq + (4 * rg + r) * (D + 4) + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = *reinterpret_cast<const float4*>(sk + (cg + 16 * e) * (D + 4) + d);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            fma_pair(s2[r][e], make_float2(a[r].x, a[r].y), make_float2(b[e].x, b[e].y));
            fma_pair(s2[r][e], make_float2(a[r].z, a[r].w), make_float2(b[e].z, b[e].w));
          }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint64_t* mrow = P.a.mask + (static_cast<int64_t>(rq.t0) + (row0 + min(4 * rg + r, rows - 1)) / P.group) * P.a.mask_words;
        float s[4], top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int u = k0 + cg + 16 * e - ctx;  // below 0: context
          const bool seen = !drafted || u < 0 || (u < rq.q_len && (__ldg(mrow + u / 64) >> (u % 64) & 1));
          s[e] = seen ? (s2[r][e].x + s2[r][e].y) * P.scale_log2 : -INFINITY;
          top = fmaxf(top, s[e]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float m_new = fmaxf(m[r], top);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;  // a row that has seen nothing yet: weights 0
        const float alpha = exp2f(m[r] - m_use);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2f(s[e] - m_use);
          sum += p;
          sp[(4 * rg + r) * (kKeys + 4) + cg + 16 * e] = p;
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[r] = l[r] * alpha + sum;
        m[r] = m_new;
#pragma unroll
        for (int c = 0; c < C; ++c) o[r][c] = make_float2(o[r][c].x * alpha, o[r][c].y * alpha);
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");  // V has landed
      __syncthreads();
      if (j + 1 < nt) stage_tile<D>(sk, kc, s_ids[(j + 1) & 1], k0 + kKeys, rq.len, head, P.hkv);
      if (drafted) add_pv<D, true>(o, sp, sv, rg, cg);
      else add_pv<D, false>(o, sp, sv, rg, cg);
      __syncthreads();
      if (j + 1 < nt) stage_tile<D>(sv, vc, s_ids[(j + 1) & 1], k0 + kKeys, rq.len, head, P.hkv);
    }
    const bool bad = s_bad != 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * rg + r;
      if (row >= rows) continue;
      float* dst;
      float f = 1.f;
      if (slot < 0) {
        const int at = row0 + row;
        dst = out + ((static_cast<int64_t>(rq.t0) + at / P.group) * A.num_q_heads + head * P.group + at % P.group) * D;
        f = l[r] == 0.f ? 0.f : 1.f / l[r];
      } else {
        const int64_t prow = static_cast<int64_t>(slot) * kRows + row;
        dst = P.part_o + prow * D;
        if (cg == 0) {
          P.part_ml[2 * prow] = m[r];
          P.part_ml[2 * prow + 1] = bad ? -1.f : l[r];
        }
      }
      const bool zero = slot < 0 && (bad || l[r] == 0.f);
#pragma unroll
      for (int c = 0; c < C; c += 2)
        *reinterpret_cast<float4*>(dst + 64 * (c / 2) + 4 * cg) =
            zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                 : make_float4(o[r][c].x * f, o[r][c].y * f, o[r][c + 1].x * f, o[r][c + 1].y * f);
    }
    __syncthreads();
  }
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_f32_merge_kernel(const Params32 P) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  join_rows<E>(
      P.cuts, P.part_o, P.part_ml, kRows, [&](const Cut& cut, int row) { return row < cut.rows[0]; },
      [&](const Cut& cut, int row, const Joined<E>& j) {
        const bool zero = j.bad || j.l == 0.f;
        const float inv = 1.f / j.l;
        const int at = cut.first[0] + row;
        float* dst = static_cast<float*>(P.a.a.out) +
                     ((static_cast<int64_t>(cut.t0) + at / P.group) * P.a.a.num_q_heads + cut.head * P.group + at % P.group) * D;
#pragma unroll
        for (int e = 0; e < E; e += 2)
          reinterpret_cast<float2*>(dst)[(lane * E + e) / 2] =
              zero ? make_float2(0.f, 0.f) : make_float2(j.o[e] * inv, j.o[e + 1] * inv);
      });
}

struct Layout32 {
  size_t o_bytes, ml_bytes, bytes;
};
Layout32 layout32(int d, int num_sms) {
  const size_t runs = static_cast<size_t>(d == 64 ? kCtasPerSm<64> : kCtasPerSm<128>) * num_sms, rows = 2 * runs * kRows;
  Layout32 l;
  l.o_bytes = rows * d * sizeof(float);
  l.ml_bytes = (rows * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255);
  l.bytes = l.o_bytes + l.ml_bytes + 2 * runs * sizeof(Cut);
  return l;
}

template <int D>
int launch_f32(const TreeArgs& t, void* workspace, int num_sms, uint32_t* err, cudaStream_t s) {
  const AttnArgs& a = t.a;
  const Layout32 l = layout32(D, num_sms);
  Params32 p{};
  p.a = t;
  p.err = err;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.o_bytes);
  p.cuts = reinterpret_cast<Cut*>(static_cast<uint8_t*>(workspace) + l.o_bytes + l.ml_bytes);
  p.hkv = a.cache.num_kv_heads;
  p.group = a.num_q_heads / p.hkv;
  p.scale_log2 = a.scale * kLog2e;
  // CTAs: as many as fit, fewer where the caller's bounds leave less to do
  const int64_t most = static_cast<int64_t>(kCtasPerSm<D>) * num_sms;
  const int64_t units = (static_cast<int64_t>(a.max_query_len) * p.group + kRows - 1) / kRows * p.hkv;
  const int64_t tiles = units >= most ? units : units * ((static_cast<int64_t>(a.max_seq_len) + kKeys - 1) / kKeys);
  const int64_t want = tiles >= most ? most : tiles * a.num_seqs;
  const int ctas = static_cast<int>(want < 1 ? 1 : want < most ? want : most);
  static uint64_t smem_set = 0;
  int st = set_smem_once(reinterpret_cast<const void*>(tree_f32_kernel<D>), kSmem32<D>, &smem_set);
  if (st) return st;
  st = cuda_status(launch_k(tree_f32_kernel<D>, dim3(ctas), dim3(kThreads), kSmem32<D>, s, p));
  if (st) return st;
  return cuda_status(launch_k(tree_f32_merge_kernel<D>, dim3(2 * ctas, 2), dim3(kMergeThreads), 0, s, p));
}

}  // namespace

int launch_tree_mask(const int32_t* parents, const int32_t* qsl, int32_t num_seqs, int64_t num_tokens, uint64_t* mask,
                     int32_t words, int32_t* depths, uint32_t* err, cudaStream_t s) {
  const int64_t blocks = (num_tokens + 127) / 128;
  if (blocks > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  return cuda_status(launch_k(tree_mask_kernel, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, s, parents, qsl,
                              num_seqs, num_tokens, mask, words, depths, err));
}

size_t tree_workspace(const pkv_cache_desc& c, int32_t num_q_heads, int32_t max_query_len, int num_sms) {
  return c.dtype == PKV_BF16 ? tree_tc_workspace(num_q_heads / c.num_kv_heads, max_query_len, num_sms)
                             : layout32(c.head_dim, num_sms).bytes;
}

int launch_tree_attention(const TreeArgs& t, void* workspace, int num_sms, uint32_t* err, cudaStream_t s) {
  if (t.a.cache.dtype == PKV_BF16) return launch_tree_tc(t, workspace, num_sms, err, s);
  return t.a.cache.head_dim == 64 ? launch_f32<64>(t, workspace, num_sms, err, s)
                                  : launch_f32<128>(t, workspace, num_sms, err, s);
}

}  // namespace pkv
