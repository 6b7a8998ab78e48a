// softmax_row.cuh -- one thread's row of a 128 x 128 score tile in TMEM: its extremum, and its
// exponents written back as bf16 P; packed fp32 arithmetic and whole-sector stores.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace pkv {

// Three-input maximum / minimum (one instruction on sm_100 and later).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// (ya, yb) = (xa, xb) * s + t and (a0, a1) += (b0, b1): one packed fp32x2 instruction
// each, rounded like the scalar forms lane by lane.
__device__ __forceinline__ void ffma2(float& ya, float& yb, float xa, float xb, float s, float t) {
  asm("{\n\t.reg .b64 x, y, m, c;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 m, {%4, %4};\n\t"
      "mov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 y, x, m, c;\n\t"
      "mov.b64 {%0, %1}, y;\n\t}"
      : "=f"(ya), "=f"(yb)
      : "f"(xa), "f"(xb), "f"(s), "f"(t));
}
__device__ __forceinline__ void fadd2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// The extremum of one S row of 128 raw scores from TMEM (taddr: the row's first
// column): the maximum, or for kPos false the minimum (a negative scale turns it into
// the maximum of scale * s).  With kMask, keys from nvis on do not count.  Each
// 32-column piece is loaded while the previous one is reduced.
template <bool kPos, bool kMask>
__device__ __forceinline__ float row_extremum(uint32_t taddr, int nvis) {
  const float hidden = kPos ? -INFINITY : INFINITY;
  float mx[8];  // eight independent running extrema keep the dependency chains short
#pragma unroll
  for (int k = 0; k < 8; ++k) mx[k] = hidden;
  uint32_t a[32], b[32];
  tmem_ld32_issue(taddr, a);
  tmem_ld32_wait(a);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t(&cur)[32] = (h & 1) ? b : a;
    uint32_t(&nxt)[32] = (h & 1) ? a : b;
    if (h < 3) tmem_ld32_issue(taddr + 32 * (h + 1), nxt);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {  // two scores per three-input instruction
      const float xa = (!kMask || 32 * h + k < nvis) ? __uint_as_float(cur[k]) : hidden;
      const float xb = (!kMask || 32 * h + k + 1 < nvis) ? __uint_as_float(cur[k + 1]) : hidden;
      const int c = (k >> 1) & 7;
      mx[c] = kPos ? fmax3(mx[c], xa, xb) : fmin3(mx[c], xa, xb);
    }
    if (h < 3) tmem_ld32_wait(nxt);
  }
  return kPos ? fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])))
              : fminf(fminf(fminf(mx[0], mx[1]), fminf(mx[2], mx[3])), fminf(fminf(mx[4], mx[5]), fminf(mx[6], mx[7])));
}

// The exponents 2^(scale * s - m_ref) of one S row (masked keys: 0, with kMask),
// written back as bf16 P over the row's first 64 columns; returns the row sum.  Each
// 32-column piece is loaded while the previous one is converted, and the 16 P columns
// a piece gives land on columns this thread has already read.  A masked key's scaled
// score is set to -inf before its exponent (an infinite raw score would give NaN at
// scale 0).  Once the P of keys 0-63 is stored, half() runs (the hand-over of that
// half) while the third piece's load is in flight.
template <bool kMask, typename Half>
__device__ __forceinline__ float row_exp_to_p(uint32_t taddr, int nvis, float scale, float m_ref, Half&& half) {
  float ls[4] = {0.f, 0.f, 0.f, 0.f};  // the row sum in four independent parts (two packed pairs)
  uint32_t a[32], b[32];
  tmem_ld32_issue(taddr, a);
  tmem_ld32_wait(a);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t(&cur)[32] = (h & 1) ? b : a;
    uint32_t(&nxt)[32] = (h & 1) ? a : b;
    if (h < 3) tmem_ld32_issue(taddr + 32 * (h + 1), nxt);
    uint32_t pw[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int k = 32 * h + 2 * q;
      float ya, yb;
      ffma2(ya, yb, __uint_as_float(cur[2 * q]), __uint_as_float(cur[2 * q + 1]), scale, -m_ref);
      const float pa = ex2_approx((!kMask || k < nvis) ? ya : -INFINITY);
      const float pb = ex2_approx((!kMask || k + 1 < nvis) ? yb : -INFINITY);
      if (q & 1) fadd2(ls[2], ls[3], pa, pb);
      else fadd2(ls[0], ls[1], pa, pb);
      __nv_bfloat162 h2 = __floats2bfloat162_rn(pa, pb);
      pw[q] = *reinterpret_cast<uint32_t*>(&h2);
    }
    tmem_st16(taddr + 16 * h, pw);
    if (h == 1) half();
    if (h < 3) tmem_ld32_wait(nxt);
  }
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

// One 32-byte global store (a whole sector) of eight 32-bit words; p is 32-byte aligned.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 32 scores to 16 columns of P; adds the weights to ls.
__device__ __forceinline__ void exp_piece(uint32_t taddr, const uint32_t (&s)[32], float scale, float m_ref,
                                          float (&ls)[4]) {
  uint32_t pw[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    float ya, yb;
    ffma2(ya, yb, __uint_as_float(s[2 * q]), __uint_as_float(s[2 * q + 1]), scale, -m_ref);
    const float pa = ex2_approx(ya), pb = ex2_approx(yb);
    if (q & 1) fadd2(ls[2], ls[3], pa, pb);
    else fadd2(ls[0], ls[1], pa, pb);
    __nv_bfloat162 h2 = __floats2bfloat162_rn(pa, pb);
    pw[q] = *reinterpret_cast<uint32_t*>(&h2);
  }
  tmem_st16(taddr, pw);
}

// row_exp_to_p without a mask in half the code: two 64-column pieces in a loop.
template <typename Half>
__device__ __forceinline__ float row_exp_to_p_loop(uint32_t taddr, float scale, float m_ref, Half&& half) {
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t a[32], b[32];
  tmem_ld32_issue(taddr, a);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    tmem_ld32_wait(a);
    tmem_ld32_issue(taddr + 64 * h + 32, b);
    exp_piece(taddr + 32 * h, a, scale, m_ref, ls);
    tmem_ld32_wait(b);
    tmem_ld32_issue(taddr + 64, a);  // (the second time for nothing)
    exp_piece(taddr + 32 * h + 16, b, scale, m_ref, ls);
    if (h == 0) half();
  }
  tmem_ld32_wait(a);
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

// The same two passes over a row whose visible keys are a bit mask: bit c of vis[c / 32] is key
// c of the tile.  These run on a request's last tiles only, and are kept small (one 32-column
// piece of code) so that they do not push the loop over its other tiles out of the
// instruction cache.  `sign` is 1, or -1 for the minimum, returned negated.
__device__ __forceinline__ float row_extremum_bits(uint32_t taddr, const uint32_t (&vis)[4], float sign) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  uint32_t v0 = vis[0], v1 = vis[1], v2 = vis[2], v3 = vis[3];
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    uint32_t a[32];
    tmem_ld32_issue(taddr + 32 * h, a);
    tmem_ld32_wait(a);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const float xa = (v0 >> k & 1u) ? __uint_as_float(a[k]) * sign : -INFINITY;
      const float xb = (v0 >> (k + 1) & 1u) ? __uint_as_float(a[k + 1]) * sign : -INFINITY;
      const int c = (k >> 1) & 3;
      mx[c] = fmax3(mx[c], xa, xb);
    }
    v0 = v1;
    v1 = v2;
    v2 = v3;
  }
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

template <typename Half>
__device__ __forceinline__ float row_exp_to_p_bits(uint32_t taddr, const uint32_t (&vis)[4], float scale, float m_ref,
                                                   Half&& half) {
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t v0 = vis[0], v1 = vis[1], v2 = vis[2], v3 = vis[3];
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    if (h == 2) half();
    uint32_t a[32];
    tmem_ld32_issue(taddr + 32 * h, a);
    tmem_ld32_wait(a);
    uint32_t pw[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float ya, yb;
      ffma2(ya, yb, __uint_as_float(a[2 * q]), __uint_as_float(a[2 * q + 1]), scale, -m_ref);
      const float pa = ex2_approx((v0 >> (2 * q) & 1u) ? ya : -INFINITY);
      const float pb = ex2_approx((v0 >> (2 * q + 1) & 1u) ? yb : -INFINITY);
      if (q & 1) fadd2(ls[2], ls[3], pa, pb);
      else fadd2(ls[0], ls[1], pa, pb);
      __nv_bfloat162 h2 = __floats2bfloat162_rn(pa, pb);
      pw[q] = *reinterpret_cast<uint32_t*>(&h2);
    }
    tmem_st16(taddr + 16 * h, pw);
    v0 = v1;
    v1 = v2;
    v2 = v3;
  }
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

}  // namespace pkv
