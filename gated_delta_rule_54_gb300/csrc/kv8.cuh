// Shared by the kernels of the 8-bit paged cache: the launch parameters and the
// conversions between bf16 / fp32 and code bytes, eight at a time.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace gdn {

struct Kv8Params {
  const __nv_bfloat16 *x, *v;  // q (attention) or k (append), and v (append)
  uint8_t* codes;
  float* scales;
  const int32_t *table, *lengths, *cu;  // lengths: start positions (append)
  __nv_bfloat16* o;
  float* lse;
  int64_t pages, rows, total;
  int64_t x_row, x_token, x_head, v_row, v_token, v_head;
  int tokens, cols, heads, group, page, causal, window;
  float scale;
};

__device__ __forceinline__ int kv8_clamp(int64_t x, int64_t lo, int64_t hi) {
  return (int)(x < lo ? lo : x > hi ? hi : x);
}

// First packed token and token count of row r (at most p.tokens; offsets that
// run backwards count as none).
__device__ __forceinline__ void kv8_row(const Kv8Params& p, int64_t r, int64_t& base, int& n) {
  if (p.cu) {
    base = p.cu[r];
    const int64_t end = p.cu[r + 1];
    n = kv8_clamp(end - base, 0, p.tokens);
    if (base < 0 || base + n > p.total) n = 0;
  } else {
    base = r * p.tokens;
    n = p.tokens;
  }
}

// Element offset of token i (of its row's n) of row r, head h in x or v.
__device__ __forceinline__ int64_t kv8_at(const Kv8Params& p, int64_t r, int64_t base, int64_t i,
                                          int64_t row, int64_t token) {
  return p.cu ? (base + i) * token : r * row + i * token;
}

__device__ __forceinline__ void bf16x8(uint4 u, float (&x)[8]) {
  float a[2];
  bf16x2(u.x, a), x[0] = a[0], x[1] = a[1];
  bf16x2(u.y, a), x[2] = a[0], x[3] = a[1];
  bf16x2(u.z, a), x[4] = a[0], x[5] = a[1];
  bf16x2(u.w, a), x[6] = a[0], x[7] = a[1];
}

// Four codes of x * rcp, little-endian (each product rounded to fp32 first).
template <int MODE>
__device__ __forceinline__ uint32_t kv8_code4(float a, float b, float c, float d, float rcp) {
  if constexpr (MODE == GDN_QDQ_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(a, rcp), __fmul_rn(b, rcp)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(c, rcp), __fmul_rn(d, rcp)), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    return (uint32_t)qdq_code<MODE>(a, rcp) | ((uint32_t)qdq_code<MODE>(b, rcp) << 8) |
           ((uint32_t)qdq_code<MODE>(c, rcp) << 16) | ((uint32_t)qdq_code<MODE>(d, rcp) << 24);
  }
}

}  // namespace gdn
