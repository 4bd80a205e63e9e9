// Logits before the beams are selected: penalties for repeated tokens, a bias, and the mask of a
// grammar.
//
// A CTA takes a slice of a row's vocabulary.  It counts the row's history into shared memory,
// where a token's place is its own, so that the same token twice meets no order; then each
// logit of the slice is read once and written once.  Eight neighbouring logits that the mask
// forbids are written without being read.  The bytes of the logits bound it.
//
// Measured on a GB300: 128 rows of 128000 bf16 logits, up to 4000 tokens said, bias and mask,
// 66 MB: 23 us, 2.8 TB/s.  A slice's chain (mask, logits, history, counts, bias) is what it waits for,
// 2.7 waves of CTAs deep: with parts left out, of then 25 us, without the history 18.5, without the bias 20, without
// the mask 21.  Counts and bias read one by one, and not in 16 bytes, took 42; logits asked for only after the
// history as well, 50.  Six CTAs of 256 threads per SM 27, 512 threads 25, 128 with eight loads 32.
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;                           // of eight logits, of a thread
constexpr int kMostSlice = 8 * kThreads * kLoads;  // tokens of a slice: their counts take 32 KB

struct LogitsParams {
  const void* logits;
  void* out;
  const int32_t *tokens, *lengths;
  const float *repetition, *frequency, *presence, *bias;
  const uint32_t* mask;
  int64_t stride, bias_row, mask_row;
  int vocab, cols, slices, slice;  // slice: a multiple of 8 * kThreads
};

__device__ __forceinline__ float load_one(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Eight neighbouring logits, aligned to 16 bytes.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    float a[2];
    bf16x2(u.x, a), x[0] = a[0], x[1] = a[1];
    bf16x2(u.y, a), x[2] = a[0], x[3] = a[1];
    bf16x2(u.z, a), x[4] = a[0], x[5] = a[1];
    bf16x2(u.w, a), x[6] = a[0], x[7] = a[1];
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// What a row's history does to the logit of a token that is in it n > 0 times; every step is
// rounded to fp32.
struct Penalty {
  float repetition, frequency, presence;
  __device__ __forceinline__ float operator()(float x, uint32_t n) const {
    x = x > 0.f ? __fdiv_rn(x, repetition) : __fmul_rn(x, repetition);
    return __fsub_rn(__fsub_rn(x, __fmul_rn(frequency, (float)n)), presence);
  }
};

// HISTORY: there are penalties.  WIDE: rows are aligned to 16 bytes.
template <typename T, bool HISTORY, bool WIDE>
__global__ void __launch_bounds__(kThreads, 5) beam_logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ uint32_t counts[];
  const int64_t row = blockIdx.x / (uint32_t)p.slices;
  const int from = (int)(blockIdx.x % (uint32_t)p.slices) * p.slice, n = min(p.slice, p.vocab - from), tid = threadIdx.x;
  const T* in = static_cast<const T*>(p.logits) + row * p.stride + from;
  T* out = static_cast<T*>(p.out) + row * p.vocab + from;
  const float* bias = p.bias ? p.bias + row * p.bias_row + from : nullptr;
  const uint32_t* mask = p.mask ? p.mask + row * p.mask_row + from / 32 : nullptr;

  // the slice's mask and logits are on their way while the history is counted
  const int wide = WIDE ? n / 8 * 8 : 0;
  uint32_t may[kLoads];
  Eight<T> x8[kLoads];
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = 8 * (tid + j * kThreads);
      may[j] = i < wide ? mask ? __ldg(mask + i / 32) >> (i % 32) & 0xffu : 0xffu : 0;
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (may[j]) x8[j].load(in + 8 * (tid + j * kThreads));
  }
  Penalty penalty = {1.f, 0.f, 0.f};
  if constexpr (HISTORY) {
    if (p.repetition) penalty.repetition = p.repetition[row];
    if (p.frequency) penalty.frequency = p.frequency[row];
    if (p.presence) penalty.presence = p.presence[row];
    const int len = p.lengths ? max(min(p.lengths[row], p.cols), 0) : p.cols;
    // eight tokens of a thread in flight, the first ones before it is known how many count
    const int32_t* said = p.tokens + row * p.cols;
    int32_t t[8];
    auto fetch = [&](int i0, int most) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = i0 + j * kThreads < most ? __ldg(said + i0 + j * kThreads) : -1;
    };
    fetch(tid, p.cols);
    for (int i = tid; i < (n + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i0 = tid; i0 < len; i0 += 8 * kThreads) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t at = (int64_t)t[j] - from;
        if (at >= 0 && at < n && i0 + j * kThreads < len) atomicAdd(&counts[at], 1u);
      }
      if (i0 + 8 * kThreads < len) fetch(i0 + 8 * kThreads, len);
    }
    __syncthreads();
  }
  auto one = [&](float x, int i) {
    if constexpr (HISTORY)
      if (const uint32_t c = counts[i]) x = penalty(x, c);
    return bias ? __fadd_rn(x, __ldg(bias + i)) : x;
  };
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = 8 * (tid + j * kThreads);
      if (i >= wide) break;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = -INFINITY;
      if (may[j]) {
        x8[j].get(x);
        if constexpr (HISTORY) {
          const uint4 c0 = *reinterpret_cast<const uint4*>(counts + i), c1 = *reinterpret_cast<const uint4*>(counts + i + 4);
          const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          if (c0.x | c0.y | c0.z | c0.w | c1.x | c1.y | c1.z | c1.w) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (c[e]) x[e] = penalty(x[e], c[e]);
          }
        }
        if (bias) {
          Eight<float> b8;
          float b[8];
          b8.load(bias + i);
          b8.get(b);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(x[e], b[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(may[j] >> e & 1)) x[e] = -INFINITY;
      }
      Eight<T>::store(out + i, x);
    }
  }
  // what is left, or all where rows are not aligned: eight of a thread in flight
  for (int i0 = wide + tid; i0 < n; i0 += 8 * kThreads) {
    float x[8];
    bool ok[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kThreads;
      ok[j] = i < n && (!mask || (__ldg(mask + i / 32) >> (i % 32) & 1));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = ok[j] ? load_one(in + i0 + j * kThreads) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kThreads;
      if (i < n) store_one(out + i, ok[j] ? one(x[j], i) : -INFINITY);
    }
  }
}

gdn_status validate_logits(const gdn_logits_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->rows < 0 || p->vocab < 1 || p->cols < 0 || (p->rows > 1 && p->stride < p->vocab)) return GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_DTYPE_BF16 && p->dtype != GDN_DTYPE_FP32)
    return p->dtype == GDN_DTYPE_FP16 ? GDN_ERR_UNSUPPORTED_DTYPE : GDN_ERR_INVALID_ARG;
  if ((p->bias_row != 0 && p->bias_row < p->vocab) || (p->mask_row != 0 && p->mask_row < ((int64_t)p->vocab + 31) / 32))
    return GDN_ERR_INVALID_ARG;
  if (p->stride > 1LL << 36 || p->rows > 0x7fffffffLL >> 8 || p->vocab > 0x7fffffff - 65536 ||
      p->cols > 0x7fffffff - 65536)  // (indices are 32-bit, some thousand ahead)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

template <typename T, bool HISTORY>
gdn_status run(const LogitsParams& q, int64_t blocks, bool wide, cudaStream_t st) {
  const size_t bytes = HISTORY ? (size_t)q.slice * 4 : 0;
  if (wide) beam_logits_kernel<T, HISTORY, true><<<(unsigned)blocks, kThreads, bytes, st>>>(q);
  else beam_logits_kernel<T, HISTORY, false><<<(unsigned)blocks, kThreads, bytes, st>>>(q);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_beam_logits_validate(const gdn_logits_problem* p) { return validate_logits(p); }

gdn_status gdn_beam_logits(const gdn_logits_problem* p, const void* logits, const int32_t* tokens,
                           const int32_t* lengths, const float* repetition, const float* frequency,
                           const float* presence, const float* bias, const int32_t* mask, void* out,
                           void* stream) {
  const gdn_status s = validate_logits(p);
  if (s != GDN_OK) return s;
  if (p->rows == 0) return GDN_OK;
  if (!logits || !out) return GDN_ERR_INVALID_ARG;
  const bool history = repetition || frequency || presence;
  if (history && !tokens && p->cols > 0) return GDN_ERR_INVALID_ARG;
  const uintptr_t elem = p->dtype == GDN_DTYPE_BF16 ? 2 : 4;
  if ((((uintptr_t)logits | (uintptr_t)out) & (elem - 1)) ||
      (((uintptr_t)tokens | (uintptr_t)lengths | (uintptr_t)repetition | (uintptr_t)frequency |
        (uintptr_t)presence | (uintptr_t)bias | (uintptr_t)mask) & 3))
    return GDN_ERR_MISALIGNED;
  // in place, or apart
  const uintptr_t a = (uintptr_t)logits, b = (uintptr_t)out;
  const int64_t stride = p->rows > 1 ? p->stride : p->vocab;
  const uintptr_t a_end = a + ((p->rows - 1) * stride + p->vocab) * elem, b_end = b + p->rows * p->vocab * elem;
  if (a < b_end && b < a_end && !(a == b && stride == p->vocab)) return GDN_ERR_INVALID_ARG;
  LogitsParams q;
  q.logits = logits, q.out = out, q.tokens = tokens, q.lengths = lengths;
  q.repetition = repetition, q.frequency = frequency, q.presence = presence, q.bias = bias;
  q.mask = reinterpret_cast<const uint32_t*>(mask);
  q.stride = stride, q.bias_row = p->bias_row, q.mask_row = p->mask_row;
  q.vocab = p->vocab, q.cols = p->cols;
  // slices that give every SM four CTAs, in steps of what a CTA writes at a time (24 x 32003 f32 2.6 us; one
  // or two 4.2 and 3.4, eight 2.6)
  constexpr int64_t kStep = 8 * kThreads;
  int64_t slice = (p->rows * p->vocab / (4 * 152) + kStep - 1) / kStep * kStep;
  q.slice = (int)(slice < kStep ? kStep : slice > kMostSlice ? kMostSlice : slice);
  q.slices = (p->vocab + q.slice - 1) / q.slice;
  const int64_t blocks = p->rows * q.slices;
  if (blocks > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
  // (128 x 128000 bf16 23 us, read one by one 56)
  const bool wide = ((a | b | (uintptr_t)bias) & 15) == 0 && p->bias_row % 4 == 0 && (p->rows == 1 || (stride * elem % 16 == 0 && p->vocab * elem % 16 == 0));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool counts = history && p->cols > 0;
  if (p->dtype == GDN_DTYPE_BF16)
    return counts ? run<__nv_bfloat16, true>(q, blocks, wide, st) : run<__nv_bfloat16, false>(q, blocks, wide, st);
  return counts ? run<float, true>(q, blocks, wide, st) : run<float, false>(q, blocks, wide, st);
}

}  // extern "C"
