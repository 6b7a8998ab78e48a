// k_tree.cu -- attention of drafted tokens, which form a tree, over an fp32 paged cache, on
// CUDA cores; and the ancestor masks of such trees.
//
// Mathematics.  Node j of request i sees the keys u < c_i = seq_len - q_len, and of the
// draft the keys c_i + b whose bit b its mask row has; out = sum_u softmax_u(scale q.K_u) V_u
// over those keys alone, with the softmax's running maximum and sum in fp32.  Keys that are
// not seen are never multiplied with anything, so whatever they hold stays out.
#include "pkv_internal.cuh"

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
// One CTA per (drafted token, kv head, chunk of up to 8 of its query heads); each warp takes
// every fourth seen key and keeps its own online-softmax state, and the four are merged at
// the end.  Lane l owns head_dim / 32 consecutive elements.
constexpr int kTreeThreads = 128;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kHeadChunk = 8;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int D>
__global__ void __launch_bounds__(kTreeThreads) tree_attention_kernel(const TreeArgs A, int64_t num_blocks, int hkv,
                                                                      float scale_log2, uint32_t* err) {
  constexpr int E = D / 32;
  __shared__ int bad;
  __shared__ float sm_m[kTreeWarps][kHeadChunk], sm_l[kTreeWarps][kHeadChunk];
  __shared__ float sm_o[kTreeWarps][kHeadChunk][D];
  grid_dep_wait();
  grid_dep_launch();
  const T* q = static_cast<const T*>(A.a.q);
  const T* kc = static_cast<const T*>(A.a.k_cache);
  const T* vc = static_cast<const T*>(A.a.v_cache);
  T* out = static_cast<T*>(A.a.out);
  const int hq = A.a.num_q_heads, group = hq / hkv;
  const int nchunks = (group + kHeadChunk - 1) / kHeadChunk;
  int64_t bid = blockIdx.x;
  const int chunk = static_cast<int>(bid % nchunks);
  bid /= nchunks;
  const int g = static_cast<int>(bid % hkv);
  const int64_t t = bid / hkv;
  const int h0 = g * group + chunk * kHeadChunk;
  const int nh = min(kHeadChunk, group - chunk * kHeadChunk);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i = find_seq(A.a.qsl, A.a.num_seqs, t);
  const int64_t q0 = __ldg(A.a.qsl + i), q1 = __ldg(A.a.qsl + i + 1);
  const int64_t L = __ldg(A.a.seq_lens + i);
  const int64_t ctx = L - (q1 - q0);
  const bool len_ok = t >= q0 && t < q1 && ctx >= 0 && (L + kBlock - 1) / kBlock <= A.a.max_blocks &&
                      q1 - q0 <= A.a.max_query_len;
  if (threadIdx.x == 0) {
    bad = len_ok ? 0 : 1;
    if (!len_ok) flag_error(err, kErrLength);
  }
  __syncthreads();
  float qr[kHeadChunk][E], m[kHeadChunk], l[kHeadChunk], o[kHeadChunk][E];
#pragma unroll
  for (int hh = 0; hh < kHeadChunk; ++hh) {
    m[hh] = -INFINITY;
    l[hh] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[hh][e] = 0.f;
      qr[hh][e] = hh < nh ? Elem<T>::to_f32(q[(t * hq + h0 + hh) * D + lane * E + e]) : 0.f;
    }
  }
  const int32_t* row = A.a.block_tables + static_cast<int64_t>(i) * A.a.max_blocks;
  const uint64_t* mrow = A.mask + t * A.mask_words;
  for (int64_t u = warp; u < (len_ok ? L : 0); u += kTreeWarps) {
    const int32_t b = __ldg(row + u / kBlock);
    if (b < 0 || b >= num_blocks) {
      if (lane == 0) {
        flag_error(err, kErrBlockId);
        bad = 1;
      }
      break;
    }
    if (u >= ctx && !(__ldg(mrow + (u - ctx) / 64) >> ((u - ctx) % 64) & 1)) continue;
    const int64_t off = ((static_cast<int64_t>(b) * hkv + g) * kBlock + u % kBlock) * D + lane * E;
    float kf[E], vf[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      kf[e] = Elem<T>::to_f32(kc[off + e]);
      vf[e] = Elem<T>::to_f32(vc[off + e]);
    }
#pragma unroll
    for (int hh = 0; hh < kHeadChunk; ++hh) {
      if (hh >= nh) break;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) dot = fmaf(qr[hh][e], kf[e], dot);
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, sh);
      const float s = dot * scale_log2;
      const float m_new = fmaxf(m[hh], s);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;  // nothing but -inf so far: weight 0
      const float alpha = exp2f(m[hh] - m_use);
      const float pr = exp2f(s - m_use);
      l[hh] = l[hh] * alpha + pr;
#pragma unroll
      for (int e = 0; e < E; ++e) o[hh][e] = fmaf(o[hh][e], alpha, pr * vf[e]);
      m[hh] = m_new;
    }
  }
#pragma unroll
  for (int hh = 0; hh < kHeadChunk; ++hh) {
    if (lane == 0) {
      sm_m[warp][hh] = m[hh];
      sm_l[warp][hh] = l[hh];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][hh][lane * E + e] = o[hh][e];
  }
  __syncthreads();
  const bool zero = bad != 0;
  for (int idx = threadIdx.x; idx < nh * D; idx += kTreeThreads) {
    const int hh = idx / D, c = idx % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kTreeWarps; ++w) M = fmaxf(M, sm_m[w][hh]);
    const float m_use = M == -INFINITY ? 0.f : M;
    float den = 0.f, num = 0.f;
#pragma unroll
    for (int w = 0; w < kTreeWarps; ++w) {
      const float f = exp2f(sm_m[w][hh] - m_use);
      den = fmaf(sm_l[w][hh], f, den);
      num = fmaf(sm_o[w][hh][c], f, num);
    }
    out[(t * hq + h0 + hh) * D + c] = Elem<T>::from_f32(zero || den == 0.f ? 0.f : num / den);
  }
}

template <typename T, int D>
int launch_typed(const TreeArgs& t, uint32_t* err, cudaStream_t s) {
  const int hkv = t.a.cache.num_kv_heads;
  const int nchunks = (t.a.num_q_heads / hkv + kHeadChunk - 1) / kHeadChunk;
  const int64_t blocks = t.a.num_tokens * hkv * nchunks;
  if (blocks > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  return cuda_status(launch_k(tree_attention_kernel<T, D>, dim3(static_cast<unsigned>(blocks)), dim3(kTreeThreads), 0,
                              s, t, t.a.cache.num_blocks, hkv, t.a.scale * kLog2e, err));
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
  return c.dtype == PKV_BF16 ? tree_tc_workspace(num_q_heads / c.num_kv_heads, max_query_len, num_sms) : 256;
}

int launch_tree_attention(const TreeArgs& t, void* workspace, int num_sms, uint32_t* err, cudaStream_t s) {
  if (t.a.cache.dtype == PKV_BF16) return launch_tree_tc(t, workspace, num_sms, err, s);
  return t.a.cache.head_dim == 64 ? launch_typed<float, 64>(t, err, s) : launch_typed<float, 128>(t, err, s);
}

}  // namespace pkv
