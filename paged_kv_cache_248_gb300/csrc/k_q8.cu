// k_q8.cu -- attention over a paged cache in 8 bits (e4m3 codes, a scale for each block and kv head).
//
// Mathematics.  With K_u = ks code_u and V_u = vs code_u, out = sum_u softmax_u(scale q.K_u) V_u over the
// keys that a query sees (causal, aligned to the context's end): one CTA a (token, query head), a key a
// thread for the scores, an element a thread for the values.
#include <cuda_fp8.h>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kKeys = 128;

struct Params {
  const __nv_bfloat16* q;
  const uint8_t *k, *v;
  const float* scales;
  const int32_t *bt, *seq_lens, *qsl;
  __nv_bfloat16* out;
  uint32_t* err;
  int64_t num_blocks, num_tokens;
  int32_t num_seqs, max_blocks, max_q, hq, hkv;
  float scale;
};

__device__ __forceinline__ float value(uint8_t x) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}

__device__ float reduce(float x, bool max) {
  __shared__ float s[4];
  for (int d = 16; d; d >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, d);
    x = max ? fmaxf(x, y) : x + y;
  }
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = max ? fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) : (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  return x;
}

__global__ void __launch_bounds__(kKeys) q8_kernel(const Params P) {
  __shared__ float qs[128], ps[kKeys];
  __shared__ int64_t rows[kKeys];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, g = h / (P.hq / P.hkv), x = threadIdx.x;
  const int i = find_seq(P.qsl, P.num_seqs, t);
  const int64_t q0 = P.qsl[i], q1 = P.qsl[i + 1], len = P.seq_lens[i], p = len - q1 + t;
  if (t < q0 || t >= q1) return;
  bool bad = q0 < 0 || q1 > P.num_tokens || q1 - q0 > P.max_q || p < 0 || len < q1 - q0 ||
             (len + kBlock - 1) / kBlock > P.max_blocks;
  if (bad && x == 0) flag_error(P.err, kErrLength);
  const int64_t at = (t * P.hq + h) * 128 + x;
  qs[x] = __bfloat162float(P.q[at]) * P.scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int64_t u0 = 0; u0 <= p && !bad; u0 += kKeys) {
    const int64_t u = u0 + x;
    float s = -INFINITY, vs = 0.f;
    bool wrong = false;
    rows[x] = -1;
    if (u <= p) {
      const int64_t id = P.bt[static_cast<int64_t>(i) * P.max_blocks + u / kBlock];
      wrong = id < 0 || id >= P.num_blocks;
      if (!wrong) {
        const float2 both = reinterpret_cast<const float2*>(P.scales)[id * P.hkv + g];
        rows[x] = ((id * P.hkv + g) * kBlock + u % kBlock) * 128;
        s = 0.f;
        for (int e = 0; e < 128; ++e) s += qs[e] * value(P.k[rows[x] + e]);
        s *= both.x;
        vs = both.y;
      }
    }
    if (__syncthreads_or(wrong)) {
      bad = true;
      if (x == 0) flag_error(P.err, kErrBlockId);
      break;
    }
    const float top = fmaxf(m, reduce(s, true));
    const float w = expf(s - top), f = expf(m - top);
    l = l * f + reduce(w, false);
    o *= f;
    m = top;
    ps[x] = w * vs;
    __syncthreads();
    for (int k = 0; k < kKeys; ++k)
      if (rows[k] >= 0) o += ps[k] * value(P.v[rows[k] + x]);
    __syncthreads();
  }
  P.out[at] = __float2bfloat16_rn(bad ? 0.f : o / l);
}

}  // namespace

size_t q8_workspace(const pkv_cache_desc&, int32_t, int32_t, int) { return 0; }

int launch_q8(const AttnArgs& a, const float* scales, void*, int, uint32_t* err, cudaStream_t s) {
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const uint8_t*>(a.k_cache);
  p.v = static_cast<const uint8_t*>(a.v_cache);
  p.scales = scales;
  p.bt = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.err = err;
  p.num_blocks = a.cache.num_blocks;
  p.num_tokens = a.num_tokens;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.max_q = a.max_query_len;
  p.hq = a.num_q_heads;
  p.hkv = a.cache.num_kv_heads;
  p.scale = a.scale;
  return cuda_status(launch_k(q8_kernel, dim3(static_cast<unsigned>(a.num_tokens), a.num_q_heads), dim3(kKeys), 0, s, p));
}

}  // namespace pkv
