// k_beam.cu -- beam search's step over the paged cache's requests: the best continuations
// of each request's beams out of their logits.
//
// Mathematics.  Beam w with token v scores cum_w + x_wv - log sum_u exp(x_wu).  Within a
// beam the order of the scores is the order of the logits, so one pass over a row can keep
// its running maximum and sum (the log-sum-exp) and its num_select best logits at once;
// only their few candidates meet the log-sum-exp, and each other, afterwards.
//
// scan_kernel.  A CTA reads a piece of one row, in chunks of 32 values a thread that stay in
// registers: each value is loaded once, feeds the thread's running sum of exponents
// (fp32, relative to the thread's running maximum), and is compared with the block's
// threshold, the num_select-th best value met so far.  Candidates carry a 64-bit key, the
// value in an order-preserving form above the complement of its index, so that all keys
// differ and equal values rank by their index.  The first threshold comes from the threads'
// maxima of the first chunk (the num_select-th best of 256 of them: at least that many values
// are as good, and only the threads with a maximum above it hold any better one), so that a
// few hundred candidates at most are ever collected from ordinary logits; when the buffer
// is full all the same (equal or rising values) it is cut down to its num_select best, the
// threshold rises, and the rest of the chunk is looked at again.
//
// select_kernel.  One CTA per request joins the pieces: the log-sum-exp of each beam in 64
// bits, then the same collection over the pieces' candidates, ranked by their 64-bit score.
//
// Bound: reading the logits once (HBM); for one request, two launches and their latency.
#include "pkv_internal.cuh"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kScanThreads = 256;
constexpr int kChunkVals = 32;                          // values of a chunk per thread
constexpr int kChunk = kScanThreads * kChunkVals;       // values of a chunk
constexpr int kMaxSelect = 64;
constexpr int kMaxBeams = 64;
constexpr int kScanCap = 1536;                          // candidates collected between cuts
constexpr int kPushMost = 4;                            // pushed per thread between barriers
constexpr int kSelThreads = 512;
constexpr int kSelCap = 2048;
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kScanCap >= kScanThreads * kPushMost + kMaxSelect, "a cut buffer takes one round of pushes");

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

// Where the values of a chunk sit: whole 16-byte vectors when every row starts on a
// 16-byte boundary (kAligned), single values of consecutive threads otherwise.  One of the
// two for all rows of a call, and counted from the row's start, so that equal rows have
// equal sums wherever they lie and their ties stay ties.
struct ScanParams {
  const void* logits;
  const uint8_t* finished;
  uint64_t* keys;    // [rows][pieces][select], best first, 0: none
  float* ml;         // [rows][pieces][2]: maximum, sum of exp(x - maximum)
  int64_t row_stride;
  int32_t vocab, select, pieces, chunks_per_piece;
};

// Cuts the `n` collected keys to the `k` best, best first in place (n >= 1).  All threads
// call it, with everything pushed; returns the new count.
template <int kThreads, int kCap>
__device__ int cut_keys(uint64_t* buf, int n, int k) {
  constexpr int kPer = (kCap + kThreads - 1) / kThreads;
  uint64_t mine[kPer];
  int rank[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x + j * kThreads;
    mine[j] = i < n ? buf[i] : 0;
    rank[j] = 0;
  }
  for (int i = 0; i < n; ++i) {  // (a broadcast read)
    const uint64_t o = buf[i];
#pragma unroll
    for (int j = 0; j < kPer; ++j) rank[j] += o > mine[j] ? 1 : 0;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < n && rank[j] < k) buf[rank[j]] = mine[j];
  }
  __syncthreads();
  return min(n, k);
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const ScanParams P) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));  // values of a 16-byte vector
  constexpr int kVecs = kChunkVals / kVec;
  __shared__ uint64_t buf[kScanCap];
  __shared__ int s_count;
  __shared__ float s_m[kScanThreads / 32], s_l[kScanThreads / 32];
  if (threadIdx.x == 0) s_count = 0;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = blockIdx.x / P.pieces;
  const int piece = static_cast<int>(blockIdx.x % P.pieces);
  if (P.finished != nullptr && __ldg(P.finished + row) != 0) return;
  const T* x = static_cast<const T*>(P.logits) + row * P.row_stride;
  float m = -INFINITY, l = 0.f;
  uint64_t floor_key = 0;  // keys up to this one are out
  // index within the row of value k of the chunk that starts at `base`
  auto index_of = [&](int64_t base, int k) -> int64_t {
    return kAligned ? base + (static_cast<int64_t>(k / kVec) * kScanThreads + threadIdx.x) * kVec + k % kVec
                    : base + static_cast<int64_t>(k) * kScanThreads + threadIdx.x;
  };
  __syncthreads();
  for (int ch = 0; ch < P.chunks_per_piece; ++ch) {
    const int64_t base = (static_cast<int64_t>(piece) * P.chunks_per_piece + ch) * kChunk;
    if (base >= P.vocab) break;
    float val[kChunkVals];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int64_t e0 = index_of(base, v * kVec);
      if (kAligned && e0 + kVec <= P.vocab) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(x + e0));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          val[v * kVec + e] = sizeof(T) == 4 ? __uint_as_float(u[e * 4 / kVec])
                                             : __uint_as_float(e & 1 ? u[e * 4 / kVec] & 0xffff0000u : u[e * 4 / kVec] << 16);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const int64_t i = index_of(base, v * kVec + e);
          val[v * kVec + e] = i < P.vocab ? Elem<T>::to_f32(x[i]) : -INFINITY;
        }
      }
    }
    float top = val[0];
#pragma unroll
    for (int k = 1; k < kChunkVals; ++k) top = fmaxf(top, val[k]);
    const float m_new = fmaxf(m, top);
    if (m_new != -INFINITY) {
      // x - m first: exact for values near the maximum, and whole for the type's lowest
      // value, which times log2(e) would not be (a NaN is no maximum, but makes the sum NaN)
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int k = 0; k < kChunkVals; k += 2) {
        a0 += ex2_approx((val[k] - m_new) * kLog2e);
        a1 += ex2_approx((val[k + 1] - m_new) * kLog2e);
      }
      l = l * ex2_approx((m - m_new) * kLog2e) + (a0 + a1);
      m = m_new;
    } else {
#pragma unroll
      for (int k = 0; k < kChunkVals; ++k) l += isnan(val[k]) ? val[k] : 0.f;
    }
    auto key_of = [&](int k) -> uint64_t {
      return (static_cast<uint64_t>(ordered_bits(val[k])) << 32) | (0xffffffffu - static_cast<uint32_t>(index_of(base, k)));
    };
    if (floor_key == 0) {
      // a threshold from the threads' maxima, ranked behind what is collected already (a
      // cut leaves room for them); the values it lets pass are collected below
      uint64_t best = 0;
#pragma unroll
      for (int k = 0; k < kChunkVals; ++k) {
        const uint64_t key = val[k] > -INFINITY ? key_of(k) : 0;
        best = key > best ? key : best;
      }
      const int had = s_count;
      __syncthreads();
      if (best != 0) buf[atomicAdd(&s_count, 1)] = best;
      __syncthreads();
      const int n = s_count - had;
      __syncthreads();
      if (threadIdx.x == 0) s_count = had;
      if (n >= P.select) {
        cut_keys<kScanThreads, kScanThreads>(buf + had, n, P.select);
        floor_key = buf[had + P.select - 1] - 1;
      }
      __syncthreads();
    }
    // collect everything better than the threshold
    uint32_t pending = 0;
    if (ordered_bits(top) >= static_cast<uint32_t>(floor_key >> 32) && top > -INFINITY) {
#pragma unroll
      for (int k = 0; k < kChunkVals; ++k)
        if (val[k] > -INFINITY && key_of(k) > floor_key) pending |= 1u << k;
    }
    while (true) {
      int pushed = 0;
#pragma unroll
      for (int k = 0; k < kChunkVals; ++k) {
        if ((pending >> k & 1u) && pushed < kPushMost) {
          const uint64_t key = key_of(k);
          if (key > floor_key) {
            buf[atomicAdd(&s_count, 1)] = key;
            ++pushed;
          }
          pending &= ~(1u << k);
        }
      }
      const int more = __syncthreads_or(pending != 0);
      const int n = s_count;
      __syncthreads();
      if (n + kScanThreads * kPushMost > kScanCap) {
        const int left = cut_keys<kScanThreads, kScanCap>(buf, n, P.select);
        if (left == P.select) floor_key = buf[P.select - 1];
        if (threadIdx.x == 0) s_count = left;
        __syncthreads();
      }
      if (!more) break;
    }
  }
  // the piece's candidates, best first
  const int n = s_count;
  __syncthreads();
  const int left = n > 0 ? cut_keys<kScanThreads, kScanCap>(buf, n, P.select) : 0;
  uint64_t* out = P.keys + (row * P.pieces + piece) * P.select;
  for (int k = threadIdx.x; k < P.select; k += kScanThreads) out[k] = k < left ? buf[k] : 0;
  // its maximum and sum
  float wm = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, d));
  if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = wm;
  __syncthreads();
  float bm = s_m[0];
#pragma unroll
  for (int w = 1; w < kScanThreads / 32; ++w) bm = fmaxf(bm, s_m[w]);
  // (a thread without values has l = 0, or NaN where it met nothing but that)
  float part = m == -INFINITY ? l : l * exp2f((m - bm) * kLog2e);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
  if ((threadIdx.x & 31) == 0) s_l[threadIdx.x >> 5] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kScanThreads / 32; ++w) sum += s_l[w];
    P.ml[(row * P.pieces + piece) * 2] = bm;
    P.ml[(row * P.pieces + piece) * 2 + 1] = sum;
  }
}

struct SelParams {
  const uint64_t* keys;
  const float* ml;
  const float* cum;
  const uint8_t* finished;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  int32_t beams, vocab, select, pieces, eos;
};

// A scored candidate: the score in its order-preserving form, then the complement of
// beam * vocab + token.
struct Cand {
  uint64_t score;
  uint32_t tie;
};
__device__ __forceinline__ bool better(const Cand& a, const Cand& b) {
  return a.score > b.score || (a.score == b.score && a.tie > b.tie);
}

// Like cut_keys, for scored candidates.
__device__ int cut_cands(uint64_t* score, uint32_t* tie, int n, int k) {
  constexpr int kPer = (kSelCap + kSelThreads - 1) / kSelThreads;
  Cand mine[kPer];
  int rank[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x + j * kSelThreads;
    mine[j] = i < n ? Cand{score[i], tie[i]} : Cand{~uint64_t(0), ~0u};
    rank[j] = 0;
  }
  for (int i = 0; i < n; ++i) {
    const Cand o{score[i], tie[i]};
#pragma unroll
    for (int j = 0; j < kPer; ++j) rank[j] += better(o, mine[j]) ? 1 : 0;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x + j * kSelThreads;
    if (i < n && rank[j] < k) {
      score[rank[j]] = mine[j].score;
      tie[rank[j]] = mine[j].tie;
    }
  }
  __syncthreads();
  return min(n, k);
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelParams P) {
  __shared__ double s_lse[kMaxBeams], s_cum[kMaxBeams];
  __shared__ uint64_t s_score[kSelCap];
  __shared__ uint32_t s_tie[kSelCap];
  __shared__ int s_count;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t n = blockIdx.x;
  const int W = P.beams;
  if (threadIdx.x == 0) s_count = 0;
  if (threadIdx.x < W) {
    const int64_t row = n * W + threadIdx.x;
    const double cum = __ldg(P.cum + row);
    s_cum[threadIdx.x] = cum;
    if (P.finished == nullptr || __ldg(P.finished + row) == 0) {
      const float* ml = P.ml + row * P.pieces * 2;
      float m = -INFINITY;
      for (int p = 0; p < P.pieces; ++p) m = fmaxf(m, __ldcg(ml + 2 * p));
      double sum = 0.0;
      for (int p = 0; p < P.pieces; ++p) {
        const float pm = __ldcg(ml + 2 * p), pl = __ldcg(ml + 2 * p + 1);
        // (a piece without values adds 0, or NaN where it met nothing but that)
        sum += pm == -INFINITY ? static_cast<double>(pl) : pl * exp(static_cast<double>(pm) - m);
      }
      s_lse[threadIdx.x] = m + log(sum);  // not finite: the beam has no candidates
    }
  }
  __syncthreads();
  const int per_beam = P.pieces * P.select;
  const int total = W * per_beam;
  Cand floor_c{0, 0};  // ordered forms of finite scores are above 0
  for (int base = 0; base < total; base += kSelThreads) {
    const int i = base + threadIdx.x;
    Cand c{0, 0};
    if (i < total) {
      const int w = i / per_beam;
      if (P.finished != nullptr && __ldg(P.finished + n * W + w) != 0) {
        if (i == w * per_beam && isfinite(s_cum[w]))
          c = Cand{ordered_bits(s_cum[w]), 0xffffffffu - (static_cast<uint32_t>(w) * P.vocab + P.eos)};
      } else {
        const uint64_t key = __ldcg(P.keys + n * total + i);
        const double lse = s_lse[w];
        const double score = s_cum[w] + (static_cast<double>(from_ordered_bits(static_cast<uint32_t>(key >> 32))) - lse);
        if (key != 0 && isfinite(lse) && isfinite(score))
          c = Cand{ordered_bits(score),
                   0xffffffffu - (static_cast<uint32_t>(w) * P.vocab + (0xffffffffu - static_cast<uint32_t>(key)))};
      }
    }
    if (better(c, floor_c)) {
      const int at = atomicAdd(&s_count, 1);
      s_score[at] = c.score;
      s_tie[at] = c.tie;
    }
    __syncthreads();
    const int cnt = s_count;
    __syncthreads();
    if (cnt + kSelThreads > kSelCap && base + kSelThreads < total) {
      const int left = cut_cands(s_score, s_tie, cnt, P.select);
      if (left == P.select) floor_c = Cand{s_score[left - 1], s_tie[left - 1]};
      if (threadIdx.x == 0) s_count = left;
      __syncthreads();
    }
  }
  const int cnt = s_count;
  __syncthreads();
  const int left = cnt > 0 ? cut_cands(s_score, s_tie, cnt, P.select) : 0;
  for (int k = threadIdx.x; k < P.select; k += kSelThreads) {
    const int64_t o = n * P.select + k;
    if (k < left) {
      const uint32_t flat = 0xffffffffu - s_tie[k];
      P.out_scores[o] = static_cast<float>(from_ordered_bits(s_score[k]));
      P.out_parents[o] = static_cast<int32_t>(flat / static_cast<uint32_t>(P.vocab));
      P.out_tokens[o] = static_cast<int32_t>(flat % static_cast<uint32_t>(P.vocab));
    } else {
      P.out_scores[o] = -INFINITY;
      P.out_parents[o] = -1;
      P.out_tokens[o] = -1;
    }
  }
}

struct BeamPlan {
  int pieces, chunks_per_piece;
  size_t key_bytes, bytes;
};

// Rows are cut into pieces until every SM has a few CTAs: a piece is at least one chunk.
BeamPlan beam_plan(int32_t num_seqs, int32_t beams, int32_t vocab, int32_t select, int num_sms) {
  const int64_t rows = static_cast<int64_t>(num_seqs) * beams;
  const int64_t chunks = (static_cast<int64_t>(vocab) + kChunk - 1) / kChunk;
  int64_t pieces = (4LL * num_sms + rows - 1) / rows;
  pieces = pieces < chunks ? (pieces < 1 ? 1 : pieces) : chunks;
  const int64_t per = (chunks + pieces - 1) / pieces;
  pieces = (chunks + per - 1) / per;
  BeamPlan b;
  b.pieces = static_cast<int>(pieces);
  b.chunks_per_piece = static_cast<int>(per);
  b.key_bytes = (static_cast<size_t>(rows) * pieces * select * sizeof(uint64_t) + 255) & ~static_cast<size_t>(255);
  b.bytes = b.key_bytes + ((static_cast<size_t>(rows) * pieces * 2 * sizeof(float) + 255) & ~static_cast<size_t>(255));
  return b;
}

}  // namespace

size_t beam_workspace(int32_t num_seqs, int32_t beams, int32_t vocab, int32_t select, int num_sms) {
  return beam_plan(num_seqs, beams, vocab, select, num_sms).bytes;
}

int launch_beam_select(const BeamArgs& a, void* workspace, int num_sms, cudaStream_t s) {
  const BeamPlan b = beam_plan(a.num_seqs, a.beams, a.vocab, a.select, num_sms);
  ScanParams p{};
  p.logits = a.logits;
  p.finished = a.finished;
  p.keys = static_cast<uint64_t*>(workspace);
  p.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + b.key_bytes);
  p.row_stride = a.row_stride;
  p.vocab = a.vocab;
  p.select = a.select;
  p.pieces = b.pieces;
  p.chunks_per_piece = b.chunks_per_piece;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.num_seqs) * a.beams * b.pieces));
  const int64_t elem = a.dtype == PKV_F32 ? 4 : 2;
  const bool aligned = (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && a.row_stride * elem % 16 == 0;
  cudaError_t e;
  if (a.dtype == PKV_F32)
    e = aligned ? launch_k(scan_kernel<float, true>, grid, dim3(kScanThreads), 0, s, p)
                : launch_k(scan_kernel<float, false>, grid, dim3(kScanThreads), 0, s, p);
  else
    e = aligned ? launch_k(scan_kernel<__nv_bfloat16, true>, grid, dim3(kScanThreads), 0, s, p)
                : launch_k(scan_kernel<__nv_bfloat16, false>, grid, dim3(kScanThreads), 0, s, p);
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  SelParams q{p.keys, p.ml, a.cum, a.finished, a.out_scores, a.out_parents, a.out_tokens,
              a.beams, a.vocab, a.select, b.pieces, a.eos};
  return cuda_status(launch_k(select_kernel, dim3(a.num_seqs), dim3(kSelThreads), 0, s, q));
}

}  // namespace pkv
