// k_append.cu -- new tokens' keys and values into the paged cache, keys (and queries) rotated by
// their positions on the way.
//
// Mathematics.  Pair (a, b) of a head's first rot_dim elements, at rotary position p, becomes
// (a cos - b sin, b cos + a sin) with row p of the table; products and differences are rounded to
// fp32 one by one, so that the result does not depend on how a compiler joins them.  A 16- or 32-bit
// cache takes the result rounded once to its type.  A cache in 8 bits holds e4m3 codes and a scale
// s for each (block, kv head), for K and V apart: value = code * s.  New scales are powers of two,
// the least with amax <= 448 s over the new rows of the block: an 8-bit float loses no more to that than
// to the exact amax / 448, and a block whose scale grows as it fills is put in the new units
// without another rounding (but for codes that leave the normal range).
//
// Work.  A row (token, head) is read as 16-byte vectors, two for each of 8 (16) lanes: the two that
// hold a vector's partners.  With 16- or 32-bit caches a CTA, or a warp, takes a token's rows.  With 8 bits the new rows of one
// (request, block, kv head, K or V) belong to a warp, up to 16 rows, 64 values a lane in registers, or with
// one token a request to eight lanes: so the scale is known before anything is written and no one else writes it.
// Request i touches at most ceil((q_i + 15) / 16) blocks, at most floor(qsl[i+1] / 16) -
// floor(qsl[i] / 16) + 2 (as many as that: two tokens in two blocks, neither number passing a multiple of 16), so block number x
// of a launch belongs to the last request with floor(qsl[i] / 16) + 2 i <= x: no plan and no prefix sum.
//
// Bound: for few tokens the launch and five loads that depend on one another (one token 2.7 us, 64 tokens 2.6 us, floor 0.2);
// for many, HBM: 5300 tokens in 8 chunks, 32 / 8 heads of 128, to 8 bits, 122 MB, 27.4 us (18.2 at the copy's rate; a CTA a token
// instead of a warp: 33.8), to bf16 26.8 (133 MB, 19.8), to fp32 48.7 (263 MB, 39.3), of 8 / 2 heads of 64 9.6 (34 MB, 5.1).
#include <cuda_fp8.h>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct Params {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, out_stride;  // elements from token to token
  const float* cos_sin;
  const int32_t* positions;
  void *k_cache, *v_cache, *q_out;
  float* scales;
  const int32_t *bt, *seq_lens, *qsl;
  uint32_t* err;
  int64_t num_tokens, num_blocks, num_angles, cache_ctas;
  int32_t num_seqs, max_blocks, max_q, hq, hkv, rot, interleaved, d;
  int32_t warp_a_token;  // else: a CTA
};

// The last request with start(i) <= x, 0 if there is none; start does not decrease.  (All lanes of a warp.)
template <typename Start>
__device__ __forceinline__ int last_request(int n, int64_t x, Start&& start) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned before = __ballot_sync(0xffffffffu, at < hi && (at == lo || start(at) <= x));
    const int part = 31 - __clz(before | 1u);
    hi = min(hi, lo + (part + 1) * step);
    lo += part * step;
  }
  return lo;
}

template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  float a[kVec], b[kVec];
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& raw, float (&x)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    x[0] = __uint_as_float(raw.x);
    x[1] = __uint_as_float(raw.y);
    x[2] = __uint_as_float(raw.z);
    x[3] = __uint_as_float(raw.w);
  } else {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[16 / sizeof(T)]) {
  unpack<T>(*reinterpret_cast<const uint4*>(p), x);
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[16 / sizeof(T)]) {
  uint4 raw;
  if constexpr (sizeof(T) == 4) {
    raw = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  *reinterpret_cast<uint4*>(p) = raw;
}

// The elements of a row that lane l holds: vectors at first() and second(), partners of one another
// where the lane's are rotated.
template <typename T>
struct Lane {
  int at, other;  // elements
  bool turns;
  int angle;  // its pairs' first column of the table

  __device__ __forceinline__ Lane(const Params& P, int l) {
    constexpr int kVec = 16 / sizeof(T);
    const int half = P.rot / 2;
    angle = l * kVec;
    if (P.interleaved || l * kVec >= half) {
      const int e = P.interleaved ? 2 * l * kVec : P.rot + 2 * (l * kVec - half);
      at = e;
      other = e + kVec;
      turns = P.interleaved && e < P.rot;
    } else {
      at = l * kVec;
      other = at + half;
      turns = true;
    }
  }
};

template <typename T>
struct Turn {
  static constexpr int kVec = 16 / sizeof(T);
  float cos[kVec], sin[kVec];

  __device__ __forceinline__ void load(const Params& P, const Lane<T>& lane, int64_t row) {
    if (!lane.turns) return;
    const float* c = P.cos_sin + row * P.rot + lane.angle;
    const float* s = c + P.rot / 2;
#pragma unroll
    for (int i = 0; i < kVec; i += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(c + i)), y = __ldg(reinterpret_cast<const float4*>(s + i));
      cos[i] = x.x, cos[i + 1] = x.y, cos[i + 2] = x.z, cos[i + 3] = x.w;
      sin[i] = y.x, sin[i + 1] = y.y, sin[i + 2] = y.z, sin[i + 3] = y.w;
    }
  }
  static __device__ __forceinline__ void pair(float& a, float& b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = x;
    b = y;
  }
  __device__ __forceinline__ void apply(const Params& P, const Lane<T>& lane, float (&a)[kVec], float (&b)[kVec]) const {
    if (!lane.turns) return;
    if (P.interleaved) {
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) {
        pair(a[2 * i], a[2 * i + 1], cos[i], sin[i]);
        pair(b[2 * i], b[2 * i + 1], cos[kVec / 2 + i], sin[kVec / 2 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) pair(a[i], b[i], cos[i], sin[i]);
    }
  }
};

// A request's tokens [t0, t1) and its context before them; false: they do not fit (flagged).
struct Request {
  int64_t t0, t1, ctx;
};
__device__ __forceinline__ bool load_request(const Params& P, int i, Request& r) {
  const int64_t q0 = __ldg(P.qsl + i), q1 = __ldg(P.qsl + i + 1), len = __ldg(P.seq_lens + i);
  r.t0 = q0;
  r.t1 = q1;
  r.ctx = len - (q1 - q0);
  return q0 >= 0 && q1 >= q0 && q1 <= P.num_tokens && q1 - q0 <= P.max_q && r.ctx >= 0 &&
         (len + kBlock - 1) / kBlock <= P.max_blocks;
}

// Token t's row of the table, -1 where it has none.
__device__ __forceinline__ int64_t angle_of(const Params& P, int64_t t, int64_t p) {
  if (P.rot == 0) return 0;
  const int64_t a = P.positions ? __ldg(P.positions + t) : p;
  return a < 0 || a >= P.num_angles ? -1 : a;
}

// Request and position of token t; false: it belongs to none that fits.
__device__ __forceinline__ bool find_token(const Params& P, int64_t t, int& i, Request& r) {
  i = last_request(P.num_seqs, t, [&](int at) { return static_cast<int64_t>(__ldg(P.qsl + at)); });
  return load_request(P, i, r);
}

// Rows first, first + step, ... of token t's queries, four of them on their way at once.
template <typename T>
__device__ __forceinline__ void rotate_q(const Params& P, int64_t t, const Lane<T>& lane, const Turn<T>& turn, bool ok, int first,
                                         int step) {
  constexpr int kAtOnce = 4;
  const T* src = static_cast<const T*>(P.q) + t * P.q_stride;
  T* dst = static_cast<T*>(P.q_out) + t * P.out_stride;
#pragma unroll 1
  for (int h0 = first; h0 < P.hq; h0 += kAtOnce * step) {
    uint4 a[kAtOnce] = {}, b[kAtOnce] = {};
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int h = h0 + k * step;
      if (!ok || h >= P.hq) continue;
      a[k] = *reinterpret_cast<const uint4*>(src + h * P.d + lane.at);
      b[k] = *reinterpret_cast<const uint4*>(src + h * P.d + lane.other);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int h = h0 + k * step;
      if (h >= P.hq) continue;
      Row<T> x;
      unpack<T>(a[k], x.a);
      unpack<T>(b[k], x.b);
      if (ok) turn.apply(P, lane, x.a, x.b);
      store_vec(dst + h * P.d + lane.at, x.a);
      store_vec(dst + h * P.d + lane.other, x.b);
    }
  }
}

// The token of this thread, and its place among the threads that share it (a CTA, or a warp where tokens are many: its
// chain of dependent loads then costs a wave of CTAs instead of several).
struct Sharer {
  int64_t token;
  int at, of;
};
__device__ __forceinline__ Sharer sharer(const Params& P, int64_t cta) {
  return P.warp_a_token ? Sharer{cta * kWarps + (threadIdx.x >> 5), static_cast<int>(threadIdx.x & 31), 32}
                        : Sharer{cta, static_cast<int>(threadIdx.x), kThreads};
}

// A cache of the inputs' type.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const Params P) {
  grid_dep_wait();
  grid_dep_launch();
  const Sharer me = sharer(P, blockIdx.x);
  const int lanes = P.d / (2 * Row<T>::kVec), group = me.at / lanes, groups = me.of / lanes;
  const Lane<T> lane(P, me.at % lanes);
  const int64_t t = me.token;
  if (t >= P.num_tokens) return;
  int i;
  Request r;
  bool ok = find_token(P, t, i, r);
  if (ok && (t < r.t0 || t >= r.t1)) return;  // behind the last request: no one's
  const int64_t p = r.ctx + t - r.t0;
  int64_t id = 0, angle = 0;
  if (!ok) {
    if (t < r.t0 || t >= r.t1) return;
    if (me.at == 0) flag_error(P.err, kErrLength);
  } else {
    id = __ldg(P.bt + static_cast<int64_t>(i) * P.max_blocks + p / kBlock);
    angle = angle_of(P, t, p);
    if (me.at == 0 && angle < 0) flag_error(P.err, kErrLength);
    if (me.at == 0 && (id < 0 || id >= P.num_blocks)) flag_error(P.err, kErrBlockId);
    ok = angle >= 0;
  }
  Turn<T> turn;
  if (ok) turn.load(P, lane, angle);
  if (P.q) rotate_q(P, t, lane, turn, ok, group, groups);
  if (!ok || id < 0 || id >= P.num_blocks) return;
  for (int row = group; row < 2 * P.hkv; row += groups) {
    const bool is_v = row >= P.hkv;
    const int h = is_v ? row - P.hkv : row;
    const T* src = is_v ? static_cast<const T*>(P.v) + t * P.v_stride : static_cast<const T*>(P.k) + t * P.k_stride;
    T* dst = static_cast<T*>(is_v ? P.v_cache : P.k_cache) + ((id * P.hkv + h) * kBlock + p % kBlock) * P.d;
    Row<T> x;
    load_vec(src + h * P.d + lane.at, x.a);
    load_vec(src + h * P.d + lane.other, x.b);
    if (!is_v) turn.apply(P, lane, x.a, x.b);
    store_vec(dst + lane.at, x.a);
    store_vec(dst + lane.other, x.b);
  }
}

// ------------------------------------------------------------------ 8 bits
__device__ __forceinline__ uint32_t finite_size(float x) {  // |x|'s bits, 0 for what is not finite
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Four codes in units `ratio` times as large.
__device__ __forceinline__ uint32_t rescale4(uint32_t x, float ratio) {
  const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xffffu), __NV_E4M3));
  const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x >> 16), __NV_E4M3));
  const float2 a = __half22float2(lo), b = __half22float2(hi);
  return e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// The least power of two s, 2^-80 at least, with amax <= 448 s (448 = 1.75 * 2^8), of amax's bits.
__device__ __forceinline__ float scale_of(uint32_t amax) {
  const int e = max(static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), -80);
  return __int_as_float((e + 127) << 23);
}

// Eight lanes' part of putting `held` rows of a block, from row `first` on in steps, into units `ratio` times as large.
__device__ __forceinline__ void rescale_rows(uint8_t* block, int first, int held, int step, float ratio) {
  for (int row = first; row < held; row += step) {
    uint4* at = reinterpret_cast<uint4*>(block + row * 128) + (threadIdx.x & 7);
    const uint4 y = *at;
    *at = make_uint4(rescale4(y.x, ratio), rescale4(y.y, ratio), rescale4(y.z, ratio), rescale4(y.w, ratio));
  }
}

__device__ __forceinline__ void store_codes(uint8_t* to, const Lane<__nv_bfloat16>& lane, float (&a)[8], float (&c)[8], float inv) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    a[k] *= inv;
    c[k] *= inv;
  }
  *reinterpret_cast<uint2*>(to + lane.at) = make_uint2(e4m3x4(a[0], a[1], a[2], a[3]), e4m3x4(a[4], a[5], a[6], a[7]));
  *reinterpret_cast<uint2*>(to + lane.other) = make_uint2(e4m3x4(c[0], c[1], c[2], c[3]), e4m3x4(c[4], c[5], c[6], c[7]));
}

// A token's queries, of CTA `cta` among those that take them.
__device__ __forceinline__ void queries8(const Params& P, int64_t cta) {
  using T = __nv_bfloat16;
  const Sharer me = sharer(P, cta);
  const int64_t t = me.token;
  if (t >= P.num_tokens) return;
  const Lane<T> lane(P, threadIdx.x & 7);
  int i;
  Request r;
  const bool ok = find_token(P, t, i, r);
  if (t < r.t0 || t >= r.t1) return;
  const int64_t angle = ok ? angle_of(P, t, r.ctx + t - r.t0) : -1;
  if (angle < 0 && me.at == 0) flag_error(P.err, kErrLength);
  Turn<T> turn;
  if (angle >= 0) turn.load(P, lane, angle);
  rotate_q(P, t, lane, turn, angle >= 0, me.at / 8, me.of / 8);
}

// A cache of e4m3 codes, d = 128, bf16 inputs, requests of one token (or none) each: CTAs [0, cache_ctas) take 16 (kv head, K or V)
// of a request's block each, eight lanes for one; the others a token's queries.  What it costs is the chain of loads (lengths,
// table, scale, row) times the waves of CTAs: a warp for each, as below, takes 3.5, 10.6, 44 and 84 us for 64, 600, 2432 and 4800
// tokens of 32 / 8 heads, this 3.2, 5.6, 14.7 and 25.8.
__global__ void __launch_bounds__(kThreads) append8_one_kernel(const Params P, int ctas_per_block) {
  using T = __nv_bfloat16;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x >= P.cache_ctas) {
    queries8(P, blockIdx.x - P.cache_ctas);
    return;
  }
  const int i = static_cast<int>(blockIdx.x / ctas_per_block);
  const int unit = static_cast<int>(blockIdx.x - static_cast<unsigned>(i) * ctas_per_block) * (kThreads / 8) + static_cast<int>(threadIdx.x >> 3);
  Request r;
  const bool fits = load_request(P, i, r);
  if (r.t0 == r.t1) return;  // (whatever its length is)
  if (!fits) {
    if (threadIdx.x == 0) flag_error(P.err, kErrLength);
    return;
  }
  const int64_t id = __ldg(P.bt + static_cast<int64_t>(i) * P.max_blocks + r.ctx / kBlock);
  const int64_t angle = angle_of(P, r.t0, r.ctx);
  if (id < 0 || id >= P.num_blocks || angle < 0) {
    if (threadIdx.x == 0) flag_error(P.err, angle < 0 ? kErrLength : kErrBlockId);
    return;
  }
  const Lane<T> lane(P, threadIdx.x & 7);
  const bool real = unit < 2 * P.hkv, is_v = unit >= P.hkv;
  const int h = !real ? 0 : is_v ? unit - P.hkv : unit, held = static_cast<int>(r.ctx % kBlock);
  float* scale = P.scales + 2 * (id * P.hkv + h) + is_v;
  const float old = real && held > 0 ? *scale : 0.f;
  const T* src = (is_v ? static_cast<const T*>(P.v) + r.t0 * P.v_stride : static_cast<const T*>(P.k) + r.t0 * P.k_stride) + h * P.d;
  float a[8] = {}, c[8] = {};
  if (real) {
    load_vec(src + lane.at, a);
    load_vec(src + lane.other, c);
  }
  if (!is_v) {
    Turn<T> turn;
    turn.load(P, lane, angle);
    turn.apply(P, lane, a, c);
  }
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) most = max(most, max(finite_size(a[e]), finite_size(c[e])));
#pragma unroll
  for (int d = 4; d; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
  __syncwarp();  // (all lanes have read the scale)
  if (!real) return;
  const float now = fmaxf(old, scale_of(most));
  uint8_t* block = static_cast<uint8_t*>(is_v ? P.v_cache : P.k_cache) + (id * P.hkv + h) * kBlock * 128;
  if (held > 0 && now != old) rescale_rows(block, 0, held, 1, old / now);
  store_codes(block + held * 128, lane, a, c, 1.f / now);
  if ((threadIdx.x & 7) == 0) *scale = now;
}

// The same for requests of any length: CTAs [0, cache_ctas) take four (block, kv head, K or V) each, a warp for one.
__global__ void __launch_bounds__(kThreads) append8_kernel(const Params P, int units_per_block) {
  using T = __nv_bfloat16;
  constexpr int kVec = 8, kRows = 4;  // rows of a warp at a time
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x >= P.cache_ctas) {
    queries8(P, blockIdx.x - P.cache_ctas);
    return;
  }
  const int lane_id = threadIdx.x & 31;
  const Lane<T> lane(P, lane_id & 7);
  const int64_t x = blockIdx.x / units_per_block;
  const int unit = static_cast<int>(blockIdx.x - x * units_per_block) * kWarps + (threadIdx.x >> 5);
  if (unit >= 2 * P.hkv) return;
  const auto start = [&](int at) { return static_cast<int64_t>(__ldg(P.qsl + at)) / kBlock + 2 * static_cast<int64_t>(at); };
  const int i = last_request(P.num_seqs, x, start);
  Request r;
  const bool fits = load_request(P, i, r);
  if (r.t0 == r.t1) return;  // (whatever its length is)
  if (!fits) {
    if (lane_id == 0) flag_error(P.err, kErrLength);
    return;
  }
  const int64_t b = r.ctx / kBlock + x - start(i);  // of the request
  const int64_t n = r.t1 - r.t0, first = b * kBlock > r.ctx ? b * kBlock : r.ctx;
  const int64_t last = (b + 1) * kBlock < r.ctx + n ? (b + 1) * kBlock : r.ctx + n;  // positions [first, last)
  if (first >= last) return;
  const int64_t id = __ldg(P.bt + static_cast<int64_t>(i) * P.max_blocks + b);
  if (id < 0 || id >= P.num_blocks) {
    if (lane_id == 0) flag_error(P.err, kErrBlockId);
    return;
  }
  const bool is_v = unit >= P.hkv;
  const int h = is_v ? unit - P.hkv : unit;
  const int rows = static_cast<int>(last - first), held = static_cast<int>(first - b * kBlock), sub = lane_id >> 3;
  float* scale = P.scales + 2 * (id * P.hkv + h) + is_v;
  const float old = held > 0 ? *scale : 0.f;
  const int64_t t0 = r.t0 + first - r.ctx;
  const T* src = (is_v ? static_cast<const T*>(P.v) + t0 * P.v_stride : static_cast<const T*>(P.k) + t0 * P.k_stride) + h * P.d;
  const int64_t stride = is_v ? P.v_stride : P.k_stride;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? P.v_cache : P.k_cache) + (id * P.hkv + h) * kBlock * 128;
  float a[kBlock / kRows][kVec], c[kBlock / kRows][kVec];
  bool there[kBlock / kRows];
  uint32_t most = 0;
#pragma unroll
  for (int g = 0; g < kBlock / kRows; ++g) {
    const int row = g * kRows + sub;
    there[g] = row < rows;
    if (there[g] && !is_v) {
      const int64_t angle = angle_of(P, t0 + row, first + row);
      there[g] = angle >= 0;
      if (!there[g]) {
        flag_error(P.err, kErrLength);
      } else {
        load_vec(src + row * stride + lane.at, a[g]);
        load_vec(src + row * stride + lane.other, c[g]);
        Turn<T> turn;
        turn.load(P, lane, angle);
        turn.apply(P, lane, a[g], c[g]);
      }
    } else if (there[g]) {
      // (a token without an angle leaves no value either: its slot stays as it is)
      there[g] = angle_of(P, t0 + row, first + row) >= 0;
      load_vec(src + row * stride + lane.at, a[g]);
      load_vec(src + row * stride + lane.other, c[g]);
    }
    if (there[g]) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) most = max(most, max(finite_size(a[g][e]), finite_size(c[g][e])));
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  const float now = fmaxf(old, scale_of(most));
  if (held > 0 && now != old) rescale_rows(dst, sub, held, kRows, old / now);
  const float inv = 1.f / now;
#pragma unroll
  for (int g = 0; g < kBlock / kRows; ++g) {
    if (there[g]) store_codes(dst + (held + g * kRows + sub) * 128, lane, a[g], c[g], inv);
  }
  __syncwarp();
  if (lane_id == 0) *scale = now;
}

}  // namespace

int launch_append(const AppendArgs& a, int num_sms, uint32_t* err, cudaStream_t s) {
  Params p{};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.out_stride = a.out_stride;
  p.cos_sin = a.cos_sin;
  p.positions = a.positions;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.q_out = a.q_out;
  p.scales = a.scales;
  p.bt = a.block_tables;
  p.seq_lens = a.seq_lens;
  p.qsl = a.qsl;
  p.err = err;
  p.num_tokens = a.num_tokens;
  p.num_blocks = a.cache.num_blocks;
  p.num_angles = a.num_angles;
  p.num_seqs = a.num_seqs;
  p.max_blocks = a.max_blocks;
  p.max_q = a.max_query_len;
  p.hq = a.q ? a.num_q_heads : 0;
  p.hkv = a.cache.num_kv_heads;
  p.rot = a.rot_dim;
  p.interleaved = a.interleaved;
  p.d = a.cache.head_dim;
  // Up to 4 tokens an SM a CTA takes one, of more tokens a warp does.  CTA and warp, 32 / 8 heads of 128 in bf16 to 8 bits: 1200 tokens
  // (4 requests of 300) 9.0 and 9.0 us, 2400 15.0 and 12.8, 5400 30.6 and 26.2; 8 / 2 heads of 64 in fp32: 64 tokens 3.6 and 3.7,
  // 1200 5.8 and 4.0, 2400 7.9 and 6.0, 5400 16.6 and 10.0
  p.warp_a_token = a.num_tokens > 4 * static_cast<int64_t>(num_sms);
  const int64_t token_ctas = p.warp_a_token ? (a.num_tokens + kWarps - 1) / kWarps : a.num_tokens;
  if (a.cache.dtype == PKV_E4M3) {
    const bool one = a.max_query_len == 1;
    const int per_cta = one ? kThreads / 8 : kWarps, ctas_per_block = (2 * p.hkv + per_cta - 1) / per_cta;
    const int64_t blocks = one ? a.num_seqs : a.num_tokens / kBlock + 2 * static_cast<int64_t>(a.num_seqs);
    p.cache_ctas = blocks * ctas_per_block;
    const int64_t ctas = p.cache_ctas + (a.q ? token_ctas : 0);
    if (ctas > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    return cuda_status(launch_k(one ? append8_one_kernel : append8_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, p,
                                ctas_per_block));
  }
  auto* kernel = a.cache.dtype == PKV_F32 ? append_kernel<float> : append_kernel<__nv_bfloat16>;
  return cuda_status(launch_k(kernel, dim3(static_cast<unsigned>(token_ctas)), dim3(kThreads), 0, s, p));
}

}  // namespace pkv
