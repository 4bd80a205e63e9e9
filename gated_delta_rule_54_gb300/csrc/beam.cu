// Beam search: selection over beams and vocabulary, and the reordering of
// states that follows it.
//
// Selection is bound by reading the logits once.  In a first launch a warp takes a
// piece of a row into registers (all its loads in flight at once), finds the
// lanes' maxima, from the k-th largest of these a bound that at least k of its
// logits reach, and then, in one more pass over the registers, the sum of
// exponentials and a bit for each of the few logits that reach it; these go into a
// list of k (one per lane, in order).  A CTA joins its eight pieces.  A second launch, of
// one CTA per batch item, joins the pieces of each beam and picks the k best
// scores of all beams.  Lists are joined by k rounds of a maximum over their
// heads.
//
// Measured on a GB300, 16 x 8 beams over 128000 bf16 logits (33 MB): 20.5 us, 1.6 TB/s,
// and 6 us; half of the issue slots are taken and DRAM waits for the instructions
// on each logit.  The first form, which kept a list logit by logit, took 63 us.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "common.cuh"
#include "launch.h"

namespace gdn {

namespace {

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
// loads of eight logits that a lane has in flight, so 2048 logits per warp; with 16,
// and the lists' code unrolled with them, 128 rows of 128000 took 77 us, with this 20 us
constexpr int kLoads = 8, kBuffer = 128;

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

// NaN counts as -inf, +inf as the largest finite number
__device__ __forceinline__ float clean(float x) {
  return fminf(fmaxf(x, -INFINITY), 3.402823466e38f);
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
  int beams, vocab, k, eos, splits;
};

// Eight logits as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void put(const float (&x)[8]) {
    u = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    float a[2];
    bf16x2(u.x, a), x[0] = a[0], x[1] = a[1];
    bf16x2(u.y, a), x[2] = a[0], x[3] = a[1];
    bf16x2(u.z, a), x[4] = a[0], x[5] = a[1];
    bf16x2(u.w, a), x[6] = a[0], x[7] = a[1];
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void put(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]), b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
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
__device__ __forceinline__ void join_warp(float& m, float& s) {
  for (int d = 16; d; d >>= 1)
    join(m, s, __shfl_xor_sync(0xffffffffu, m, d), __shfl_xor_sync(0xffffffffu, s, d));
}

// The k largest keys of 32 descending lists, one per lane (next(i): the lane's
// i-th key, 0 past its end): lane i returns the i-th.
template <typename F>
__device__ __forceinline__ uint64_t merge_lists(int k, int lane, F next) {
  uint64_t head = next(0), out = 0;
  int at = 0;
  for (int r = 0; r < k; ++r) {
    const uint32_t hi = (uint32_t)(head >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t low = __reduce_max_sync(0xffffffffu, hi == top ? (uint32_t)head : 0u);
    const uint64_t best = ((uint64_t)top << 32) | low;
    if (lane == r) out = best;
    if (best != 0 && head == best) head = next(++at);
  }
  return out;
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads) beam_slice_kernel(const SelectParams p) {
  __shared__ float2 red[kSelWarps];
  __shared__ uint64_t best[kSelWarps][32];
  __shared__ uint64_t buffer[kSelWarps][kBuffer];  // candidates of a warp on their way to its list
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t row = blockIdx.x / p.splits;
  const int split = blockIdx.x % p.splits;
  if (p.finished && p.finished[row]) return;
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  const int i0 = (split * kSelWarps + warp) * (256 * kLoads) + lane * 8;
  // rows whose start is not on 16 bytes are read one element at a time
  const bool vec = ((uintptr_t)x & 15) == 0;
  Eight<T> raw[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int i = i0 + j * 256;
    if (vec && i + 8 <= p.vocab) {
      raw[j].load(x + i);
    } else {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < p.vocab ? Eight<T>::one(x + i + e) : -INFINITY;
      raw[j].put(v);
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    float v[8];
    raw[j].get(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, v[e]);  // (a NaN leaves it as it is)
  }
  m = clean(m);
  // the k-th largest of the lanes' maxima: at least k logits of the piece reach it
  float bound = -INFINITY;
  {
    uint32_t mine = (uint32_t)(order_key(m, 0) >> 32);
    uint32_t top = 0;
    for (int r = 0; r < p.k; ++r) {
      top = __reduce_max_sync(0xffffffffu, mine);
      const unsigned who = __ballot_sync(0xffffffffu, mine == top);
      if (lane == __ffs(who) - 1) mine = 0;
    }
    if (top) bound = key_value((uint64_t)top << 32);
  }
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float mu = m == -INFINITY ? 0.f : m;
  // candidates: the logits that reach the bound, as a bit per logit of the lane.
  // Where less than k lanes hold a finite one, these are the finite ones, and of
  // the others the first k in order of their index lie in the first 64 places.
  const float least = fmaxf(bound, -3.402823466e38f);
  float s = 0.f;
  uint64_t in = 0;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    float v[8];
    raw[j].get(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = clean(v[e]);
      s += ex2_approx_f((v[e] - mu) * kLog2eF);
      if (v[e] >= least) in |= 1ull << (8 * j + e);
      if (j == 0 && bound == -INFINITY && lane < 8 && v[e] == -INFINITY && i0 + e < p.vocab) in |= 1ull << e;
    }
  }
  uint64_t list = 0, kth = 0;
  int held = 0;  // keys in the warp's buffer
  auto flush = [&]() {
    __syncwarp();
    for (int i = 0; i < held; ++i) {
      const uint64_t c = buffer[warp][i];
      if (c > kth) {
        list_insert(list, c, lane);
        kth = __shfl_sync(0xffffffffu, list, p.k - 1);
      }
    }
    held = 0;
    __syncwarp();
  };
  for (unsigned who; (who = __ballot_sync(0xffffffffu, in != 0)) != 0;) {
    if (held + 32 > kBuffer) flush();
    if (in) {
      const int bit = __ffsll(in) - 1;
      const int i = i0 + (bit >> 3) * 256 + (bit & 7);
      const float c = clean(Eight<T>::one(x + i)) + 0.f;  // (again from memory: it is near)
      buffer[warp][held + __popc(who & ((1u << lane) - 1))] = order_key(c, (uint32_t)i);
      in &= in - 1;
    }
    held += __popc(who);
  }
  flush();
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (lane == 0) red[warp] = make_float2(m, s);
  best[warp][lane] = list;
  __syncthreads();
  if (warp != 0) return;
  const float2 st = lane < kSelWarps ? red[lane] : make_float2(-INFINITY, 0.f);
  m = st.x, s = st.y;
  join_warp(m, s);
  list = merge_lists(p.k, lane, [&](int i) { return lane < kSelWarps && i < p.k ? best[lane][i] : 0ull; });
  const int64_t at = row * p.splits + split;
  if (lane == 0) p.stats[at] = make_float2(m, s);
  if (lane < p.k) p.keys[at * p.k + lane] = list;
}

__global__ void __launch_bounds__(1024) beam_join_kernel(const SelectParams p) {
  __shared__ uint64_t cand[32][32];  // [beam][rank]: score, beam and rank as one key
  __shared__ float score[32][32];
  __shared__ int32_t token[32][32];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;  // one warp per beam
  const int64_t item = blockIdx.x, row = item * p.beams + w;
  const float given = p.scores[row], before = given == given ? given : -INFINITY;
  const bool done = p.finished && p.finished[row];
  grid_dep_wait();
  float sc = -INFINITY;
  int32_t tk = done ? p.eos : 0;
  if (done) {
    if (lane == 0) sc = before;
  } else {
    float m = -INFINITY, s = 0.f;
    uint64_t list = 0;
    // 31 pieces at a time; the last lane brings what is there already
    for (int i0 = 0; i0 < p.splits; i0 += 31) {
      const int64_t at = row * p.splits + i0 + lane;
      const bool have = lane < 31 && i0 + lane < p.splits;
      const float2 st = have ? p.stats[at] : make_float2(-INFINITY, 0.f);
      float m2 = st.x, s2 = st.y;
      join_warp(m2, s2);
      join(m, s, m2, s2);
      cand[w][lane] = list;
      __syncwarp();
      list = merge_lists(p.k, lane, [&](int i) {
        return i >= p.k ? 0ull : have ? p.keys[at * p.k + i] : lane == 31 ? cand[w][i] : 0ull;
      });
      __syncwarp();
    }
    if (list) {
      tk = (int32_t)key_index(list);
      if (m > -INFINITY) sc = __fadd_rn(__fsub_rn(key_value(list), m), __fsub_rn(before, logf(s)));
    }
  }
  cand[w][lane] = order_key(sc + 0.f, (uint32_t)(w * 32 + lane));
  score[w][lane] = sc;
  token[w][lane] = tk;
  __syncthreads();
  if (w != 0) return;
  const uint64_t list = merge_lists(p.k, lane, [&](int i) {
    return lane < p.beams && i < p.k ? cand[lane][i] : 0ull;
  });
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
  if (p->batch * p->beams > 0x1ffffff || p->vocab > (1 << 30)) return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

int splits_of(const gdn_beam_problem& p) {
  constexpr int64_t piece = (int64_t)kSelThreads * 8 * kLoads;
  return (int)((p.vocab + piece - 1) / piece);
}

// ---------------------------------------------------------------------------
// Reorder.  A thread owns one 16-byte column of all rows of a group of beams: it
// loads the rows that some other row takes and then stores, so the same kernel
// works in place, and a row that keeps itself costs nothing there.
// 16 x 8 beams, two layers of 1 MiB each, into other buffers: 58 us for 268 MB
// written and at most as many read; HBM bounds it (71 % busy).
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

// The states go through one launch in no order, so no buffer that is written may meet
// another one, but for a state's own in place.  Buffers in the order of their addresses:
// a written one must lie past all before it, a read one past all written ones (the same
// buffer may be read for several states).
bool apart(int n, const void* const* src, void* const* dst, const int64_t* row_bytes,
           const int32_t* parents, int64_t rows) {
  struct Range {
    uintptr_t from, to;
    bool written;
  };
  Range few[128], *r = few;
  std::unique_ptr<Range[]> many;
  if (2 * (int64_t)n + 1 > 128) {
    many.reset(new (std::nothrow) Range[2 * (size_t)n + 1]);
    if (!(r = many.get())) return false;
  }
  int64_t m = 0;
  r[m++] = {(uintptr_t)parents, (uintptr_t)(parents + rows), false};
  for (int i = 0; i < n; ++i) {
    if (row_bytes[i] == 0) continue;
    const uintptr_t a = (uintptr_t)src[i], c = (uintptr_t)dst[i], bytes = (uintptr_t)(rows * row_bytes[i]);
    r[m++] = {c, c + bytes, true};
    if (a != c) r[m++] = {a, a + bytes, false};
  }
  std::sort(r, r + m, [](const Range& x, const Range& y) { return x.from < y.from; });
  uintptr_t any = 0, written = 0;
  for (int64_t i = 0; i < m; ++i) {
    if (r[i].from < (r[i].written ? any : written)) return false;
    any = std::max(any, r[i].to);
    if (r[i].written) written = std::max(written, r[i].to);
  }
  return true;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_beam_validate(const gdn_beam_problem* p) { return validate_beam(p); }

size_t gdn_beam_workspace_bytes(const gdn_beam_problem* p) {
  if (validate_beam(p) != GDN_OK) return 0;
  return (size_t)(p->batch * p->beams) * splits_of(*p) * 8 * (1 + (size_t)p->k);
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
  q.splits = splits_of(*p);
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
  }
  if (!apart(n, src, dst, row_bytes, parents, rows)) return GDN_ERR_INVALID_ARG;
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
