// The 8-bit paged cache: append, and the entry points of append and attention.
#include <math.h>

#include "kv8.cuh"
#include "launch.h"

namespace gdn {

namespace {

// Append.  A CTA takes a touched page of a row and some of its 2 * heads blocks (K
// and V of a head): the new tokens of a block are read once into registers (CH
// chunks of eight bf16 per thread, the next block's while this one is worked on),
// their maximum is the block's, and their codes go out as 8-byte stores.  The
// bytes are the bf16 tokens in and the codes out; the old codes of the page are
// read and written only when the new tokens raise its scale.  A NaN or an infinity
// makes the scale one, and the block's codes mean nothing then.  Eight uneven prompts of
// up to 4096 tokens, 8 heads of 128, pages of 32, INT8, 121 MB: 22.5 us, 5.4 TB/s
// (28 us before the next block's loads were in flight).
template <int MODE, int DIM, int NT, int CH>
__global__ void __launch_bounds__(NT) kv8_append_kernel(const Kv8Params p, int blocks, int per) {
  constexpr int C8 = DIM / 8;
  __shared__ float red[2][NT / 32];
  const int64_t r = blockIdx.x / blocks;
  const int tid = threadIdx.x;
  int64_t base;
  int n;
  kv8_row(p, r, base, n);
  const int64_t st = p.lengths[r];
  if (st < 0) return;
  const int64_t b = (st >> p.shift) + blockIdx.x % blocks;
  const int64_t lo = st > b * p.page ? st : b * p.page;
  const int64_t hi = st + n < (b + 1) * p.page ? st + n : (b + 1) * p.page;
  if (lo >= hi || b >= p.cols) return;
  const int64_t id = p.table[r * p.cols + b];
  if (id < 0 || id >= p.pages) return;
  const int64_t xat = kv8_at(p, r, base, lo - st, p.x_row, p.x_token);
  const int64_t vat = kv8_at(p, r, base, lo - st, p.v_row, p.v_token);
  const int chunks = (int)(hi - lo) * C8, old = (int)(lo - b * p.page);
  const int first = blockIdx.y * per, last = min(first + per, 2 * p.heads);

  // block i: head i / 2, K or V
  auto tile_of = [&](int i) { return ((i & 1) * p.pages + id) * p.heads + i / 2; };
  auto load = [&](int i, uint4 (&u)[CH], float& was) {
    const __nv_bfloat16* x = i & 1 ? p.v + vat + (i / 2) * p.v_head : p.x + xat + (i / 2) * p.x_head;
    const int64_t step = i & 1 ? p.v_token : p.x_token;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * NT;
      u[j] = make_uint4(0, 0, 0, 0);
      if (c < chunks) u[j] = __ldg(reinterpret_cast<const uint4*>(x + (c / C8) * step + (c % C8) * 8));
    }
    was = old > 0 ? p.scales[tile_of(i)] : 0.f;
  };
  uint4 next[CH];
  float next_was;
  load(first, next, next_was);
  for (int i = first; i < last; ++i) {
    uint4 u[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) u[j] = next[j];
    const float was = next_was;
    if (i + 1 < last) load(i + 1, next, next_was);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      float f[8];
      bf16x8(u[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(f[e]));
    }
    m = warp_max(m);  // (of bit patterns: a NaN, which max_nan gives without sign, is above all)
    if constexpr (NT > 32) {
      float(&part)[NT / 32] = red[i & 1];
      if (tid % 32 == 0) part[tid / 32] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) m = max_nan(m, part[w]);
    } else {
      __syncwarp();  // every lane has read the block's scale
    }
    float now = max_nan(was, __fdiv_rn(m, QdqMax<MODE>::value)), rcp = __frcp_rn(now);
    if (isinf(rcp)) now = rcp = 0.f;

    const int64_t tile = tile_of(i);
    uint8_t* out = p.codes + tile * p.page * DIM;
    if (now > was) {
      for (int c = tid; c < old * C8; c += NT) {
        const uint2 w = *reinterpret_cast<const uint2*>(out + c * 8);
        const float4 a = qdq_code4_values<MODE>(w.x), e = qdq_code4_values<MODE>(w.y);
        *reinterpret_cast<uint2*>(out + c * 8) =
            make_uint2(kv8_code4<MODE>(__fmul_rn(a.x, was), __fmul_rn(a.y, was),
                                       __fmul_rn(a.z, was), __fmul_rn(a.w, was), rcp),
                       kv8_code4<MODE>(__fmul_rn(e.x, was), __fmul_rn(e.y, was),
                                       __fmul_rn(e.z, was), __fmul_rn(e.w, was), rcp));
      }
    }
    if (tid == 0 && (now != was || old == 0)) p.scales[tile] = now;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = tid + j * NT;
      if (c < chunks) {
        float f[8];
        bf16x8(u[j], f);
        *reinterpret_cast<uint2*>(out + (old * C8 + c) * 8) = make_uint2(
            kv8_code4<MODE>(f[0], f[1], f[2], f[3], rcp), kv8_code4<MODE>(f[4], f[5], f[6], f[7], rcp));
      }
    }
  }
}

template <int MODE, int DIM>
gdn_status run_append(const Kv8Params& p, cudaStream_t st) {
  // pages that n consecutive positions can touch
  const int blocks = (p.tokens + p.page - 2) / p.page + 1;
  if (p.rows * blocks > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
  // blocks per CTA, whose loads overlap: up to 8 while 152 SMs still get eight CTAs
  // each (8 prompts to 4096 tokens 23.4 us, with one block each 28.8; one such
  // prompt, which gives less CTAs, 6.4 and 6.2)
  int per = 1;
  while (per < 8 && per < 2 * p.heads && p.rows * blocks * 2 * p.heads / (2 * per) >= 152 * 8) per *= 2;
  const dim3 grid((unsigned)(p.rows * blocks), (unsigned)((2 * p.heads + per - 1) / per));
  const int chunks = (p.tokens < p.page ? p.tokens : p.page) * (DIM / 8);
  if (chunks <= 32)
    kv8_append_kernel<MODE, DIM, 32, 1><<<grid, 32, 0, st>>>(p, blocks, per);
  else if (chunks <= 128)
    kv8_append_kernel<MODE, DIM, 128, 1><<<grid, 128, 0, st>>>(p, blocks, per);
  else if (chunks <= 512)
    kv8_append_kernel<MODE, DIM, 128, 4><<<grid, 128, 0, st>>>(p, blocks, per);
  else
    kv8_append_kernel<MODE, DIM, 256, 8><<<grid, 256, 0, st>>>(p, blocks, per);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status validate_kv8(const gdn_kv8_problem* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->pages < 0 || p->rows < 0 || p->total < 0 || p->tokens < 0 || p->cols < 0 ||
      p->heads <= 0 || p->group <= 0 || p->window < 0 || (p->causal != 0 && p->causal != 1))
    return GDN_ERR_INVALID_ARG;
  if (p->mode != GDN_QDQ_E4M3 && p->mode != GDN_QDQ_INT8)
    return p->mode == GDN_QDQ_NONE ? GDN_ERR_UNSUPPORTED_MODE : GDN_ERR_INVALID_ARG;
  if (p->dtype != GDN_DTYPE_BF16) {
    if (p->dtype == GDN_DTYPE_FP16 || p->dtype == GDN_DTYPE_FP32) return GDN_ERR_UNSUPPORTED_DTYPE;
    return GDN_ERR_INVALID_ARG;
  }
  if (p->dim != 64 && p->dim != 128) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if (!p->cu_seqlens && p->total != p->rows * p->tokens) return GDN_ERR_INVALID_ARG;
  if (p->rows == 0 && p->total > 0) return GDN_ERR_INVALID_ARG;
  // positions are 32-bit, with room to round one up to a tile of keys and to look some
  // tiles ahead; heads are a grid dimension; page ids are 32-bit
  if ((int64_t)p->cols * p->page > 0x7fff0000LL || p->pages > 0x7fffffffLL ||
      p->rows > 0x7fffffffLL || p->total > 0x7fffffffLL ||
      2 * p->pages * p->heads > 0x7fffffffLL || p->rows * p->heads > 0x7fffffffLL ||
      (int64_t)p->tokens * p->group > 0x7ffffeffLL || (int64_t)p->heads * p->group > 65535)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if (!isfinite(p->scale)) return GDN_ERR_INVALID_ARG;
  for (const int64_t s : {p->x_row, p->x_token, p->x_head, p->v_row, p->v_token, p->v_head})
    if (s % 8 != 0) return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

Kv8Params params_of(const gdn_kv8_problem& p) {
  Kv8Params k = {};
  k.pages = p.pages, k.rows = p.rows, k.total = p.total;
  k.x_row = p.x_row, k.x_token = p.x_token, k.x_head = p.x_head;
  k.v_row = p.v_row, k.v_token = p.v_token, k.v_head = p.v_head;
  k.tokens = p.tokens, k.cols = p.cols, k.heads = p.heads, k.group = p.group, k.page = p.page;
  k.shift = __builtin_ctz((unsigned)p.page);
  k.causal = p.causal, k.window = p.window, k.scale = p.scale;
  k.cu = p.cu_seqlens;
  return k;
}

// One 16-row tile holds a row's queries of a K/V head: the kernel that streams the
// codes, else the one that converts them for tiles of 128 rows.  Measured with
// 16 query rows, stream / tiles in us: 64 rows x 8 heads, 8192 keys each, 128-wide E4M3
// 245/358, INT8 209/401, 64-wide 164/288 and 155/310 (four query rows, 128-wide: 178/358
// and 190/401); 1 x 8 x 700 keys 13.9/13.2, 12.7/13.2, 10.1/11.3 and 9.7/11.7.  A full
// wave of short keys, 16 x 8 x 2048: 25/30, 22/31, 17/24 and 16/24.
bool few_rows(const gdn_kv8_problem& p) { return (int64_t)p.tokens * p.group <= 16; }

bool off16(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if ((uintptr_t)q & 15) return true;
  return false;
}
bool off4(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if ((uintptr_t)q & 3) return true;
  return false;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_kv8_validate(const gdn_kv8_problem* p) { return validate_kv8(p); }

size_t gdn_kv8_workspace_bytes(const gdn_kv8_problem* p) {
  if (validate_kv8(p) != GDN_OK) return 0;
  return few_rows(*p) ? kv8_decode_workspace(params_of(*p), p->dim)
                      : kv8_prefill_workspace(params_of(*p), p->dim);
}

gdn_status gdn_kv8_append(const gdn_kv8_problem* p, const void* k, const void* v, uint8_t* codes,
                          float* scales, const int32_t* table, const int32_t* start,
                          void* stream) {
  const gdn_status s = validate_kv8(p);
  if (s != GDN_OK) return s;
  if (p->total == 0 || p->pages == 0 || p->cols == 0 || p->tokens == 0) return GDN_OK;
  if (!k || !v || !codes || !scales || !table || !start) return GDN_ERR_INVALID_ARG;
  if (off16({k, v, codes}) || off4({scales, table, start, p->cu_seqlens}))
    return GDN_ERR_MISALIGNED;
  Kv8Params prm = params_of(*p);
  prm.x = static_cast<const __nv_bfloat16*>(k);
  prm.v = static_cast<const __nv_bfloat16*>(v);
  prm.codes = codes, prm.scales = scales, prm.table = table, prm.lengths = start;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p->mode == GDN_QDQ_E4M3)
    return p->dim == 128 ? run_append<GDN_QDQ_E4M3, 128>(prm, st)
                         : run_append<GDN_QDQ_E4M3, 64>(prm, st);
  return p->dim == 128 ? run_append<GDN_QDQ_INT8, 128>(prm, st)
                       : run_append<GDN_QDQ_INT8, 64>(prm, st);
}

gdn_status gdn_kv8_attention(const gdn_kv8_problem* p, const void* q, const uint8_t* codes,
                             const float* scales, const int32_t* table, const int32_t* lengths,
                             void* o, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const gdn_status s = validate_kv8(p);
  if (s != GDN_OK) return s;
  if (p->total == 0) return GDN_OK;
  if (!q || !o || !lengths) return GDN_ERR_INVALID_ARG;
  // (the kernels look up a row's pages whether or not the cache has any)
  if (p->cols > 0 && (!table || (p->pages > 0 && (!codes || !scales)))) return GDN_ERR_INVALID_ARG;
  if (off16({q, codes, o}) || off4({scales, table, lengths, lse, p->cu_seqlens}) ||
      ((uintptr_t)workspace & 255))
    return GDN_ERR_MISALIGNED;
  const size_t need = gdn_kv8_workspace_bytes(p);
  if (workspace_bytes < need || (need > 0 && !workspace)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  Kv8Params prm = params_of(*p);
  prm.x = static_cast<const __nv_bfloat16*>(q);
  prm.codes = const_cast<uint8_t*>(codes), prm.scales = const_cast<float*>(scales);
  prm.table = table, prm.lengths = lengths;
  prm.o = static_cast<__nv_bfloat16*>(o), prm.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few_rows(*p)) return launch_kv8_decode(prm, p->mode, p->dim, workspace, st);
  return launch_kv8_prefill(prm, p->mode, p->dim, workspace, st);
}

}  // extern "C"
