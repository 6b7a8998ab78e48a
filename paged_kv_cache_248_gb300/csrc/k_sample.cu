// k_sample.cu -- tokens drawn from logits, with temperature, top-k, min-p and top-p.
//
// Mathematics.  The candidates of a row in order (larger logit first, of equal ones the lower index) have the
// weights w = exp((x - max) / T).  Every filter keeps a beginning of that order: the first k; those with
// w >= min_p; the shortest with mass >= top_p of what is left.  The token is the first whose cumulative
// weight exceeds u times the kept mass.  Whether a sum of a hundred thousand weights lies above or below
// a border is decided by its last digits, so weights are whole numbers: w 2^S rounded, right to about 2^-40
// of w (weight() below), and sums of them exact, in any order.
#include "pkv_internal.cuh"
#include "weight.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 1024;

struct Params {
  const void* logits;
  int64_t stride;
  const float *temperature, *top_p, *min_p, *uniform;
  const int32_t* top_k;
  int32_t* tokens;
  float* logprobs;
  uint32_t* err;
  int32_t vocab, shift;
};

template <typename T>
__device__ __forceinline__ float load(const Params& P, int64_t row, int i) {
  return Elem<T>::to_f32(static_cast<const T*>(P.logits)[row * P.stride + i]);
}

// Larger logits have smaller keys; the index in the lower half.
__device__ __forceinline__ uint64_t key_of(float x, int i) {
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  const uint32_t up = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<uint64_t>(~up) << 32 | static_cast<uint32_t>(i);
}

// Candidates with keys of at most `key`: how many, and their mass.
template <typename T>
__device__ void upto(const Params& P, int64_t row, uint64_t key, const Weight& w, const uint64_t* table, uint64_t* count,
                     uint64_t* mass) {
  __shared__ unsigned long long s[2];
  if (threadIdx.x == 0) s[0] = s[1] = 0;
  __syncthreads();
  unsigned long long n = 0, m = 0;
  for (int i = threadIdx.x; i < P.vocab; i += kThreads) {
    const float x = load<T>(P, row, i);
    if (isfinite(x) && key_of(x, i) <= key) {
      ++n;
      m += w.of(x, table);
    }
  }
  atomicAdd(&s[0], n);
  atomicAdd(&s[1], m);
  __syncthreads();
  *count = s[0];
  *mass = s[1];
  __syncthreads();
}

// The least key for which enough(count, mass) holds.
template <typename T, typename Enough>
__device__ uint64_t least(const Params& P, int64_t row, const Weight& w, const uint64_t* table, Enough&& enough) {
  uint64_t lo = 0, hi = ~uint64_t(0);
  while (lo < hi) {
    const uint64_t mid = lo + (hi - lo) / 2;
    uint64_t n, m;
    upto<T>(P, row, mid, w, table, &n, &m);
    if (enough(n, m)) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const Params P) {
  __shared__ unsigned long long s_first;
  __shared__ uint64_t table[256];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = blockIdx.x;
  if (threadIdx.x < 256) table[threadIdx.x] = kPowers.v[threadIdx.x];
  if (threadIdx.x == 0) s_first = ~0ull;
  __syncthreads();
  unsigned long long first = ~0ull;
  for (int i = threadIdx.x; i < P.vocab; i += kThreads) {
    const float x = load<T>(P, row, i);
    if (isfinite(x)) first = min(first, static_cast<unsigned long long>(key_of(x, i)));
  }
  atomicMin(&s_first, first);
  __syncthreads();
  const float temp = P.temperature ? P.temperature[row] : 1.f, u = P.uniform[row];
  const float top_p = P.top_p ? P.top_p[row] : 1.f, min_p = P.min_p ? P.min_p[row] : 0.f;
  const int32_t top_k = P.top_k ? P.top_k[row] : 0;
  const bool wrong = !(temp >= 0.f && temp <= 3.4e38f) || !(u >= 0.f && u < 1.f) || !(top_p >= 0.f) || !(min_p <= 1.f);
  if (wrong || s_first == ~0ull) {
    if (threadIdx.x == 0) {
      if (wrong) flag_error(P.err, kErrSetting);
      P.tokens[row] = -1;
      if (P.logprobs) P.logprobs[row] = -INFINITY;
    }
    return;
  }
  const int best = static_cast<int>(s_first & 0xffffffffu);
  if (temp == 0.f) {
    if (threadIdx.x == 0) {
      P.tokens[row] = best;
      if (P.logprobs) P.logprobs[row] = 0.f;
    }
    return;
  }
  const Weight w(load<T>(P, row, best), temp, P.shift);
  uint64_t all, mass, cut = ~uint64_t(0), n;
  upto<T>(P, row, cut, w, table, &all, &mass);
  if (top_k > 0 && static_cast<uint64_t>(top_k) < all)
    cut = least<T>(P, row, w, table, [&](uint64_t c, uint64_t) { return c >= static_cast<uint64_t>(top_k); });
  if (min_p > 0.f) {
    // the first candidate whose weight is below: one less is kept
    __shared__ unsigned long long s_low;
    if (threadIdx.x == 0) s_low = ~0ull;
    __syncthreads();
    const uint64_t least_w = w.part_up(min_p);
    for (int i = threadIdx.x; i < P.vocab; i += kThreads) {
      const float x = load<T>(P, row, i);
      if (isfinite(x) && w.of(x, table) < least_w) atomicMin(&s_low, static_cast<unsigned long long>(key_of(x, i)));
    }
    __syncthreads();
    if (s_low - 1 < cut) cut = s_low - 1;
    __syncthreads();
  }
  upto<T>(P, row, cut, w, table, &n, &mass);
  if (top_p < 1.f) {
    const uint64_t want = part_of_up(mass, top_p);
    const uint64_t end = least<T>(P, row, w, table, [&](uint64_t c, uint64_t m) { return c >= 1 && m >= want; });
    if (end < cut) cut = end;
    upto<T>(P, row, cut, w, table, &n, &mass);
  }
  const uint64_t target = part_of(mass, u);
  const uint64_t key = least<T>(P, row, w, table, [&](uint64_t, uint64_t m) { return m > target; });
  if (threadIdx.x == 0) {
    const int token = static_cast<int>(key & 0xffffffffu);
    P.tokens[row] = token;
    if (P.logprobs) P.logprobs[row] = w.log_share(load<T>(P, row, token), table, mass);
  }
}

}  // namespace

int launch_sample(const SampleArgs& a, int, uint32_t* err, cudaStream_t s) {
  Params p{a.logits, a.row_stride, a.temperature, a.top_p, a.min_p, a.uniform, a.top_k, a.tokens, a.logprobs, err, a.vocab,
           weight_shift(a.vocab)};
  auto* kernel = a.dtype == PKV_F32 ? sample_kernel<float> : sample_kernel<__nv_bfloat16>;
  return cuda_status(launch_k(kernel, dim3(a.num_seqs), dim3(kThreads), 0, s, p));
}

}  // namespace pkv
