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
  int tokens, cols, heads, group, page, shift, causal, window;  // page == 1 << shift
  float scale;
};

// Keys of a row that any of its queries sees: positions [begin, end).
struct Kv8Span {
  int64_t base;     // first packed token (queries)
  int n, len;       // queries, tokens
  int begin, end;
};

__device__ __forceinline__ int kv8_clamp(int64_t x, int64_t lo, int64_t hi) {
  return (int)(x < lo ? lo : x > hi ? hi : x);
}

// First packed token and token count of row r (at most p.tokens; offsets that
// run backwards count as none).  False where a packed row has more tokens than that, or
// lies outside of the call's.
__device__ __forceinline__ bool kv8_row(const Kv8Params& p, int64_t r, int64_t& base, int& n) {
  if (p.cu) {
    base = p.cu[r];
    const int64_t end = p.cu[r + 1];
    n = kv8_clamp(end - base, 0, p.tokens);
    if (base < 0 || base + n > p.total) n = 0;
    return end - base <= n;
  }
  base = r * p.tokens;
  n = p.tokens;
  return true;
}

// Element offset of token i (of its row's n) of row r, head h in x or v.
__device__ __forceinline__ int64_t kv8_at(const Kv8Params& p, int64_t r, int64_t base, int64_t i,
                                          int64_t row, int64_t token) {
  return p.cu ? (base + i) * token : r * row + i * token;
}

__device__ __forceinline__ Kv8Span kv8_span(const Kv8Params& p, int64_t r) {
  Kv8Span s;
  if (!kv8_row(p, r, s.base, s.n)) s.n = 0;
  s.len = p.lengths[r];
  const int64_t first = (int64_t)s.len - s.n;  // position of the first query
  s.end = kv8_clamp(s.len, 0, (int64_t)p.cols * p.page);
  s.begin = p.window > 0 ? kv8_clamp(first - p.window + 1, 0, s.end) : 0;
  if (s.n == 0) s.begin = s.end = 0;
  return s;
}

// Keys that query i of the row sees: [begin, end).
__device__ __forceinline__ void kv8_seen(const Kv8Params& p, const Kv8Span& s, int i, int& begin,
                                         int& end) {
  const int64_t pos = (int64_t)s.len - s.n + i;
  end = p.causal ? kv8_clamp(pos + 1, 0, s.end) : pos < 0 ? 0 : s.end;
  begin = p.window > 0 ? kv8_clamp(pos - p.window + 1, 0, s.end) : 0;
}

// Packed calls: outputs that no row computes, written by warp w of all.  Tokens before the
// first row and after the last one belong to no query: 0 and -inf.  A row that breaks the
// call's bound (kv8_row) gets NaN.
template <int DIM>
__device__ __forceinline__ void kv8_fill(const Kv8Params& p, int64_t w, int64_t all, int lane) {
  const int64_t width = p.heads * p.group;
  auto fill = [&](int64_t t0, int64_t t1, uint32_t pair, float lse) {
    t0 = t0 < 0 ? 0 : t0, t1 = t1 > p.total ? p.total : t1;
    for (int64_t i = t0 * width + w; i < t1 * width; i += all) {
      if (lane < DIM / 8) reinterpret_cast<uint4*>(p.o + i * DIM)[lane] = make_uint4(pair, pair, pair, pair);
      if (p.lse && lane == 0) p.lse[i] = lse;
    }
  };
  fill(0, p.cu[0], 0u, -INFINITY);
  fill(p.cu[p.rows], p.total, 0u, -INFINITY);
  for (int64_t r0 = 0; r0 < p.rows; r0 += 32) {
    int64_t base;
    int n;
    unsigned over = __ballot_sync(0xffffffffu, r0 + lane < p.rows && !kv8_row(p, r0 + lane, base, n));
    for (; over; over &= over - 1) {
      const int64_t r = r0 + __ffs(over) - 1;
      fill(p.cu[r], p.cu[r + 1], 0x7fff7fffu, __int_as_float(0x7fffffff));
    }
  }
}

// Code bytes to fp16 pairs: of the bytes b0 b1 b2 b3 of w, even = (b0, b2) and
// odd = (b1, b3).  An E4M3 byte s eeee mmm moved to the fp16 fields reads
// value * 2^-8, subnormals included, and exactly; no byte gives an infinity or
// NaN, so what lies in slots without a token (weight 0) cannot spoil a sum.  An
// INT8 byte c is 1024 + (c + 128) in fp16 less 1152, exactly.
template <int MODE>
__device__ __forceinline__ void kv8_half2(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (MODE == GDN_QDQ_E4M3) {
    even = ((w << 8) & 0x80008000u) | ((w << 7) & 0x3f803f80u);
    odd = (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u);
  } else {
    const uint32_t e = (w & 0x00ff00ffu) ^ 0x64806480u, o = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&e), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&o), off);
    even = *reinterpret_cast<const uint32_t*>(&a);
    odd = *reinterpret_cast<const uint32_t*>(&b);
  }
}
// what kv8_half2 leaves out of the value, as a power of two
template <int MODE>
constexpr float kKv8Shift = MODE == GDN_QDQ_E4M3 ? 8.f : 0.f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// maximum that is NaN where an operand is
__device__ __forceinline__ float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// A power of two that brings a row of q with this largest magnitude to [2^E, 2^(E+1)),
// and its inverse.  Where that is an infinity the power is 0, which makes a NaN of it, and
// of every score of the row (8 bits hold no infinity).  (In fp16 with E = 8 a row's
// small elements keep at least 33 bits below its largest.)
template <int E>
__device__ __forceinline__ void kv8_q_factor(float most, float& to, float& back) {
  int e = (int)(__float_as_uint(most) >> 23) - 127;
  e = e < -118 ? -118 : e > 127 ? 127 : e;  // both powers are normal numbers
  to = most <= 3.402823466e38f ? __uint_as_float((uint32_t)(E - e + 127) << 23) : 0.f;
  back = __uint_as_float((uint32_t)(e - E + 127) << 23);
}

// q beside E4M3 codes.  A row with its largest element in [2^7, 2^8) is the sum of an E4M3
// number (four bits) and what that leaves (at most 2^-4 of an element's binade, so three of
// bf16's eight bits) as an E5M2 number: exact for elements down to 2^-13 of the largest.
// Below 2^-6 the first is off by at most 2^-10, of which three bits leave 2^-14, i.e. such
// elements are off by at most 2^-21 of the row's largest.  (INT8 codes meet q in fp16,
// which is exact down to 2^-25 of it.)  Four codes at a time, little-endian.
__device__ __forceinline__ uint32_t kv8_q_first(const float* f, float to, float (&rest)[4]) {
  float2 a, b;
  const uint32_t w = e4m3_code2(f[0], f[1], to, a) | (uint32_t)e4m3_code2(f[2], f[3], to, b) << 16;
  rest[0] = f[0] * to - a.x, rest[1] = f[1] * to - a.y;
  rest[2] = f[2] * to - b.x, rest[3] = f[3] * to - b.y;
  return w;
}
__device__ __forceinline__ uint32_t kv8_e5m2x4(const float (&x)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E5M2);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E5M2);
  return lo | hi << 16;
}
__device__ __forceinline__ void mma_e5m2_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The scales of a block as the kernels take them: K's, and log2 of V's.  Where one of the
// two is no number in [0, inf) K's is NaN, so that the scores, and what comes of them, are
// NaN for the queries that see a key of the block, and for no others.
__device__ __forceinline__ float2 kv8_scales(float ks, float vs) {
  const float top = 3.402823466e38f;
  if (!(ks >= 0.f && ks <= top && vs >= 0.f && vs <= top)) return make_float2(__int_as_float(0x7fffffff), -INFINITY);
  return make_float2(ks, lg2_approx(vs));
}

// What turns a query's sum over P V into its output: 2^(mv - m) / l, in two steps, since the
// power by itself may lie below the normal numbers.  0 where no key is seen (l is 0) or every V
// scale seen is 0 (mv is -inf), NaN where a score is (l is NaN).
template <int MODE>
__device__ __forceinline__ float kv8_out_factor(float mv, float m, float l) {
  if (l == 0.f) return 0.f;
  if (mv == -INFINITY) return 0.f * l;
  const float half = ex2_approx_f(0.5f * (mv - m + kKv8Shift<MODE>));
  return half * (half / l);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
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
    // |x rcp| is at most 127 (1 + 2^-22) where rcp comes from a scale of at least
    // max |x| / 127, so no clamp is needed; adding 1.5 * 2^23 rounds to the nearest
    // integer, ties to even, which is then the low byte
    constexpr float kInt = 12582912.f;
    const uint32_t i0 = __float_as_uint(__fmul_rn(a, rcp) + kInt), i1 = __float_as_uint(__fmul_rn(b, rcp) + kInt);
    const uint32_t i2 = __float_as_uint(__fmul_rn(c, rcp) + kInt), i3 = __float_as_uint(__fmul_rn(d, rcp) + kInt);
    return __byte_perm(__byte_perm(i0, i1, 0x0040), __byte_perm(i2, i3, 0x0040), 0x5410);
  }
}

// What an append with rotation has besides: the queries, and the angles of the positions.
struct Kv8Rotary {
  const __nv_bfloat16* q;
  const float *cos, *sin;
  int64_t positions, q_row, q_token, q_head;
  int dim, interleaved;
};

// Launchers (arguments validated).
gdn_status launch_kv8_rotary(const Kv8Params& p, const Kv8Rotary& w, int mode, int dim,
                             cudaStream_t st);
size_t kv8_shared_workspace(const Kv8Params& p, int beams, int dim);
gdn_status launch_kv8_shared(const Kv8Params& p, int beams, const int32_t* shared, int mode, int dim,
                             void* workspace, cudaStream_t st);
size_t kv8_decode_workspace(const Kv8Params& p, int dim);
gdn_status launch_kv8_decode(const Kv8Params& p, int mode, int dim, void* workspace,
                             cudaStream_t st);
size_t kv8_prefill_workspace(const Kv8Params& p, int dim);
gdn_status launch_kv8_prefill(const Kv8Params& p, int mode, int dim, void* workspace,
                              cudaStream_t st);
int kv8_prefill_device_error(bool reset);
int kv8_shared_device_error(bool reset);

}  // namespace gdn
