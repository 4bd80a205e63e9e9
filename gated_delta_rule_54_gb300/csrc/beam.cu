// Beam search: selection over beams and vocabulary, and the reordering of
// states that follows it.
//
// Selection is bound by reading the logits once.  A first launch gives each
// slice of a row to one CTA: in one pass over the slice it keeps the running
// maximum and sum of exponentials of the log-softmax and, per warp, the K best
// logits (one per lane, in order; a logit below the K-th is dropped by one
// comparison).  A second, of one CTA per batch item, joins the slices of each
// beam and picks the K best scores of all beams.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace gdn {

namespace {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;

// Order of (value, index): larger value first, then lower index.  The value's
// bits are mapped so that they order as integers; no key of a value is 0.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t index) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return ((uint64_t)o << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint32_t key_index(uint64_t k) { return ~(uint32_t)k; }

// Puts key c (the same in every lane) into the warp's list, one key per lane
// in descending order; what falls off lane 31 is dropped.
__device__ __forceinline__ void list_insert(uint64_t& list, uint64_t c, int lane) {
  const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
  if (list < c) list = lane > 0 && up < c ? up : c;
}

// NaN counts as -inf, +inf as the largest finite number; -0 as +0
__device__ __forceinline__ float clean(float x) {
  return x == x ? fminf(x, 3.402823466e38f) + 0.f : -INFINITY;
}

struct SelectParams {
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  float* scores_out;
  int32_t *parents, *tokens;
  uint8_t* finished_out;
  uint64_t* keys;  // workspace: [batch * beams, splits, k] best logits of a slice
  float2* stats;   // workspace: [batch * beams, splits] maximum, sum of exp(x - maximum)
  int64_t stride;
  int beams, vocab, k, eos, splits, slice;
};

template <typename T>
struct Load8;
template <>
struct Load8<__nv_bfloat16> {
  static __device__ __forceinline__ void vec(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    float a[2];
    bf16x2(u.x, a), x[0] = a[0], x[1] = a[1];
    bf16x2(u.y, a), x[2] = a[0], x[3] = a[1];
    bf16x2(u.z, a), x[4] = a[0], x[5] = a[1];
    bf16x2(u.w, a), x[6] = a[0], x[7] = a[1];
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Load8<float> {
  static __device__ __forceinline__ void vec(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};

// (m, s) of the union of two sets, each as its maximum and its sum of exp(x - maximum)
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  if (top == -INFINITY) return;
  s = s * expf(m - top) + s2 * expf(m2 - top);
  m = top;
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads) beam_slice_kernel(const SelectParams p) {
  __shared__ float2 red[kSelWarps];
  __shared__ uint64_t best[kSelWarps][32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t row = blockIdx.x / p.splits;
  const int split = blockIdx.x % p.splits;
  if (p.finished && p.finished[row]) return;
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  const int begin = split * p.slice, end = min(begin + p.slice, p.vocab);
  // rows whose start is not on 16 bytes are read one element at a time
  const bool vec = ((uintptr_t)x & 15) == 0;
  float m = -INFINITY, s = 0.f;
  uint64_t list = 0;
  float least = -INFINITY;  // a logit below this is not among the warp's K best
  for (int i0 = begin + warp * 256; i0 < end; i0 += kSelWarps * 256) {
    const int i = i0 + lane * 8;
    float v[8];
    const int left = end - i;
    if (vec && left >= 8) {
      Load8<T>::vec(x + i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = clean(v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < left ? clean(Load8<T>::one(x + i + j)) : -INFINITY;
    }
    float top = v[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, v[j]);
    if (top > m) s *= expf(m - top), m = top;
    if (m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s += expf(v[j] - m);
    }
    unsigned lanes = __ballot_sync(0xffffffffu, left > 0 && top >= least);
    while (lanes) {
      const int from = __ffs(lanes) - 1;
      lanes &= lanes - 1;
      const int n = min(__shfl_sync(0xffffffffu, left, from), 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = __shfl_sync(0xffffffffu, v[j], from);
        if (j < n && c >= least) {
          list_insert(list, order_key(c, (uint32_t)(i0 + from * 8 + j)), lane);
          const uint64_t kth = __shfl_sync(0xffffffffu, list, p.k - 1);
          least = kth ? key_value(kth) : -INFINITY;
        }
      }
    }
  }
  for (int d = 16; d; d >>= 1)
    join(m, s, __shfl_xor_sync(0xffffffffu, m, d), __shfl_xor_sync(0xffffffffu, s, d));
  if (lane == 0) red[warp] = make_float2(m, s);
  best[warp][lane] = list;
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < kSelWarps; ++w) {
    join(m, s, red[w].x, red[w].y);
    for (int j = 0; j < p.k; ++j) {
      const uint64_t c = best[w][j];
      if (c <= __shfl_sync(0xffffffffu, list, p.k - 1)) break;
      list_insert(list, c, lane);
    }
  }
  const int64_t at = row * p.splits + split;
  if (lane == 0) p.stats[at] = make_float2(m, s);
  if (lane < p.k) p.keys[at * p.k + lane] = list;
}

__global__ void __launch_bounds__(1024) beam_join_kernel(const SelectParams p) {
  __shared__ float score[32][32];  // [beam][rank]
  __shared__ int32_t token[32][32];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;  // one warp per beam
  const int64_t item = blockIdx.x, row = item * p.beams + w;
  grid_dep_wait();
  const float before = p.scores[row];
  const bool done = p.finished && p.finished[row];
  float sc = -INFINITY;
  int32_t tk = done ? p.eos : 0;
  if (done) {
    if (lane == 0) sc = before;
  } else {
    float m = -INFINITY, s = 0.f;
    uint64_t list = 0;
    for (int i = 0; i < p.splits; ++i) {
      const float2 st = p.stats[row * p.splits + i];
      join(m, s, st.x, st.y);
      const uint64_t mine = lane < p.k ? p.keys[(row * p.splits + i) * p.k + lane] : 0;
      for (int j = 0; j < p.k; ++j) {
        const uint64_t c = __shfl_sync(0xffffffffu, mine, j);
        if (c <= __shfl_sync(0xffffffffu, list, p.k - 1)) break;
        list_insert(list, c, lane);
      }
    }
    if (list) {
      tk = (int32_t)key_index(list);
      if (m > -INFINITY) sc = __fadd_rn(__fsub_rn(key_value(list), m), __fsub_rn(before, logf(s)));
    }
  }
  score[w][lane] = sc;
  token[w][lane] = tk;
  __syncthreads();
  if (w != 0) return;
  uint64_t list = 0;
  for (int b = 0; b < p.beams; ++b) {
    const uint64_t mine = order_key(score[b][lane], (uint32_t)(b * 32 + lane));
    for (int j = 0; j < p.k; ++j) {
      const uint64_t c = __shfl_sync(0xffffffffu, mine, j);
      if (c <= __shfl_sync(0xffffffffu, list, p.k - 1)) break;
      list_insert(list, c, lane);
    }
  }
  if (lane < p.k) {
    const int at = (int)key_index(list), b = at / 32, t = token[b][at % 32];
    const int64_t out = item * p.k + lane;
    p.scores_out[out] = score[b][at % 32];
    p.parents[out] = (int32_t)(item * p.beams + b);
    p.tokens[out] = t;
    p.finished_out[out] = (p.finished && p.finished[item * p.beams + b]) || (p.eos >= 0 && t == p.eos);
  }
}

gdn_status validate_beam(const gdn_beam_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->batch < 0 || p->vocab <= 0 || p->stride < p->vocab) return GDN_ERR_INVALID_ARG;
  if (p->beams < 1 || p->beams > 32 || p->k < 1 || p->k > 32) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (p->dtype != GDN_DTYPE_BF16 && p->dtype != GDN_DTYPE_FP32)
    return p->dtype == GDN_DTYPE_FP16 ? GDN_ERR_UNSUPPORTED_DTYPE : GDN_ERR_INVALID_ARG;
  if (p->eos < -1 || p->eos >= p->vocab) return GDN_ERR_INVALID_ARG;
  if (p->batch * p->beams > 0x1ffffff) return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

// Slices of a row: enough CTAs to fill 152 SMs four times over, of at least
// 4096 logits (two loads of 8 per thread)
void slices_of(const gdn_beam_problem& p, int& splits, int& slice) {
  const int64_t rows = p.batch * p.beams;
  const int64_t want = rows > 0 ? (152 * 4 + rows - 1) / rows : 1;
  const int64_t most = (p.vocab + 4095) / 4096;
  int64_t n = want < most ? want : most;
  if (n < 1) n = 1;
  slice = (int)(((p.vocab + n - 1) / n + 2047) / 2048 * 2048);
  splits = (p.vocab + slice - 1) / slice;
}

// ---------------------------------------------------------------------------
// Reorder.  A thread owns one 16-byte column of all rows of a group of beams: it
// loads the rows that some other row takes and then stores, so the same kernel
// works in place, and a row that keeps itself costs nothing there.
// ---------------------------------------------------------------------------
constexpr int kMaxStates = 64, kReorderThreads = 256;

struct ReorderParams {
  const uint4* src[kMaxStates];
  uint4* dst[kMaxStates];
  int64_t vecs[kMaxStates];    // 16-byte vectors of a row
  int64_t first[kMaxStates + 1];  // first block of each state
  const int32_t* parents;
  int64_t rows;
  int n, beams;
};

template <int W>
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  int i = 0;
  while (i + 1 < p.n && (int64_t)blockIdx.x >= p.first[i + 1]) ++i;
  const int64_t b = blockIdx.x - p.first[i], vecs = p.vecs[i];
  const int64_t per = (vecs + kReorderThreads - 1) / kReorderThreads;
  const int64_t group = b / per, col = b % per * kReorderThreads + threadIdx.x;
  const int64_t r0 = group * p.beams;
  const int n = (int)(p.rows - r0 < p.beams ? p.rows - r0 : p.beams);
  if (col >= vecs) return;
  const uint4* src = p.src[i];
  uint4* dst = p.dst[i];
  const bool in_place = src == dst;
  uint4 u[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < n) {
      int64_t q = p.parents[r0 + w];
      if (in_place && (q < r0 || q >= r0 + n) && q != -1) q = r0 + w;
      const bool load = q >= 0 && q < p.rows && !(in_place && q == r0 + w);
      u[w] = load ? src[q * vecs + col] : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < n) {
      int64_t q = p.parents[r0 + w];
      if (in_place && (q < r0 || q >= r0 + n) && q != -1) q = r0 + w;
      if (!(in_place && q == r0 + w)) dst[(r0 + w) * vecs + col] = u[w];
    }
  }
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_beam_validate(const gdn_beam_problem* p) { return validate_beam(p); }

size_t gdn_beam_workspace_bytes(const gdn_beam_problem* p) {
  if (validate_beam(p) != GDN_OK) return 0;
  int splits, slice;
  slices_of(*p, splits, slice);
  return (size_t)(p->batch * p->beams) * splits * 8 * (1 + (size_t)p->k);
}

gdn_status gdn_beam_select(const gdn_beam_problem* p, const void* logits, const float* scores,
                           const uint8_t* finished, float* scores_out, int32_t* parents,
                           int32_t* tokens, uint8_t* finished_out, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const gdn_status s = validate_beam(p);
  if (s != GDN_OK) return s;
  if (p->batch == 0) return GDN_OK;
  if (!logits || !scores || !scores_out || !parents || !tokens || !finished_out)
    return GDN_ERR_INVALID_ARG;
  const uintptr_t elem = p->dtype == GDN_DTYPE_BF16 ? 1 : 3;
  if (((uintptr_t)logits & elem) || ((uintptr_t)workspace & 15) ||
      (((uintptr_t)scores | (uintptr_t)scores_out | (uintptr_t)parents | (uintptr_t)tokens) & 3))
    return GDN_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < gdn_beam_workspace_bytes(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  SelectParams q;
  q.logits = logits, q.scores = scores, q.finished = finished, q.scores_out = scores_out;
  q.parents = parents, q.tokens = tokens, q.finished_out = finished_out;
  q.stride = p->stride, q.beams = p->beams, q.vocab = p->vocab, q.k = p->k, q.eos = p->eos;
  slices_of(*p, q.splits, q.slice);
  const int64_t rows = p->batch * p->beams, blocks = rows * q.splits;
  if (blocks > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
  q.stats = static_cast<float2*>(workspace);
  q.keys = reinterpret_cast<uint64_t*>(q.stats + blocks);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p->dtype == GDN_DTYPE_BF16)
    beam_slice_kernel<__nv_bfloat16><<<(unsigned)blocks, kSelThreads, 0, st>>>(q);
  else
    beam_slice_kernel<float><<<(unsigned)blocks, kSelThreads, 0, st>>>(q);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p->batch);
  cfg.blockDim = dim3(32 * p->beams);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_join_kernel, q) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_beam_reorder(int32_t n, const void* const* src, void* const* dst,
                            const int64_t* row_bytes, const int32_t* parents, int64_t rows,
                            int32_t beams, void* stream) {
  if (n < 0 || rows < 0 || beams < 1) return GDN_ERR_INVALID_ARG;
  if (beams > 32) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (n == 0 || rows == 0) return GDN_OK;
  if (!src || !dst || !row_bytes || !parents) return GDN_ERR_INVALID_ARG;
  if ((uintptr_t)parents & 3) return GDN_ERR_MISALIGNED;
  for (int i = 0; i < n; ++i) {
    if (row_bytes[i] < 0) return GDN_ERR_INVALID_ARG;
    if (row_bytes[i] % 16 != 0) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (row_bytes[i] == 0) continue;
    if (!src[i] || !dst[i]) return GDN_ERR_INVALID_ARG;
    if (((uintptr_t)src[i] | (uintptr_t)dst[i]) & 15) return GDN_ERR_MISALIGNED;
    const uintptr_t a = (uintptr_t)src[i], c = (uintptr_t)dst[i], bytes = (uintptr_t)(rows * row_bytes[i]);
    if (a != c && a < c + bytes && c < a + bytes) return GDN_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t groups = (rows + beams - 1) / beams;
  for (int i = 0; i < n;) {
    ReorderParams p;
    p.parents = parents, p.rows = rows, p.beams = beams, p.n = 0;
    int64_t blocks = 0;
    for (; i < n && p.n < kMaxStates; ++i) {
      if (row_bytes[i] == 0) continue;
      const int64_t vecs = row_bytes[i] / 16;
      const int64_t add = groups * ((vecs + kReorderThreads - 1) / kReorderThreads);
      if (add > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
      if (blocks + add > 0x7fffffffLL) break;
      p.src[p.n] = static_cast<const uint4*>(src[i]);
      p.dst[p.n] = static_cast<uint4*>(dst[i]);
      p.vecs[p.n] = vecs;
      p.first[p.n] = blocks;
      blocks += add;
      ++p.n;
    }
    if (p.n == 0) break;
    p.first[p.n] = blocks;
    if (beams <= 4) beam_reorder_kernel<4><<<(unsigned)blocks, kReorderThreads, 0, st>>>(p);
    else if (beams <= 8) beam_reorder_kernel<8><<<(unsigned)blocks, kReorderThreads, 0, st>>>(p);
    else if (beams <= 16) beam_reorder_kernel<16><<<(unsigned)blocks, kReorderThreads, 0, st>>>(p);
    else beam_reorder_kernel<32><<<(unsigned)blocks, kReorderThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  return GDN_OK;
}

}  // extern "C"
