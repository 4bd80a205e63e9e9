// The 8-bit paged cache: append with the rotation of queries and keys on the way.
//
// Pair j of a head's first 2 * half dims (dims j and j + half, or 2 j and 2 j + 1) turns by
// the angle of the token's position, in fp32 with every product rounded:
//     a' = fl(fl(a cos) - fl(b sin)),   b' = fl(fl(b cos) + fl(a sin))
// The turned keys are quantized as they are, without a rounding to bf16 between; queries are
// rounded to bf16 and go to an array of their own.
//
// A thread holds units of 16 elements: the two chunks of eight whose elements are each
// other's partners (or two neighbouring chunks, where pairs are neighbours or nothing turns), so
// that a pair meets in registers.  Its angles stay there while it goes through the heads of
// its token.  The bytes of q, k, v and the codes bound it.
//
// Measured on a GB300: eight uneven prompts of up to 4096 tokens, 8 K/V heads of 128 and 32 query
// heads, E4M3, 446 MB: 88 us, 5.1 TB/s (copying: 6.8), DRAM and issue (0.51 a clock and scheduler)
// together, two CTAs of 123 registers per SM.  With 512 threads of one unit each 124, or 112 with two
// such CTAs per SM; 256 of two units with three CTAs per SM 143, with four 161; 128 of four units 90.
// 64 single tokens: 2.7 us, launch and latency.
#include <math.h>

#include "kv8.cuh"
#include "launch.h"

namespace gdn {

namespace {

struct RotaryParams {
  Kv8Params p;  // x, v: keys and values; o: queries out
  const __nv_bfloat16* q;
  const float *cos, *sin;  // [positions, half]
  int64_t positions, q_row, q_token, q_head;
  int half, inter;
};

// Where unit u of a head lies: its two chunks of eight elements, and whether it turns.
struct Unit {
  int c0, c1;
  bool turns;
};
__device__ __forceinline__ Unit unit_of(const RotaryParams& a, int u) {
  const bool turns = u < a.half / 8, apart = turns && !a.inter;
  return {apart ? u : 2 * u, apart ? u + a.half / 8 : 2 * u + 1, turns};
}

// cos and sin of a unit's eight pairs; NaN at a position that the tables do not have.
__device__ __forceinline__ void angles(const RotaryParams& a, int64_t pos, int u, float (&c)[8], float (&s)[8]) {
  if (pos >= 0 && pos < a.positions) {
    const float4* pc = reinterpret_cast<const float4*>(a.cos + pos * a.half + 8 * u);
    const float4* ps = reinterpret_cast<const float4*>(a.sin + pos * a.half + 8 * u);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(pc + i), y = __ldg(ps + i);
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s[i] = __int_as_float(0x7fffffff);
  }
}

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float a = x, b = y;
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
__device__ __forceinline__ void turn16(float (&lo)[8], float (&hi)[8], const float (&c)[8], const float (&s)[8], bool inter) {
  if (inter) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turn(lo[2 * e], lo[2 * e + 1], c[e], s[e]);
      turn(hi[2 * e], hi[2 * e + 1], c[4 + e], s[4 + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) turn(lo[e], hi[e], c[e], s[e]);
  }
}

__device__ __forceinline__ float most16(const float (&lo)[8], const float (&hi)[8], float m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max_nan(m, max_nan(fabsf(lo[e]), fabsf(hi[e])));
  return m;
}
template <int MODE>
__device__ __forceinline__ uint2 code8(const float (&x)[8], float rcp) {
  return make_uint2(kv8_code4<MODE>(x[0], x[1], x[2], x[3], rcp), kv8_code4<MODE>(x[4], x[5], x[6], x[7], rcp));
}
__device__ __forceinline__ uint4 bf16x8_of(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Scale and its reciprocal of a block whose new tokens' largest magnitude is m.
template <int MODE>
__device__ __forceinline__ float block_scale(float was, float m, float& rcp) {
  const float now = max_nan(was, __fdiv_rn(m, QdqMax<MODE>::value));
  rcp = __frcp_rn(now);
  if (isinf(rcp)) return rcp = 0.f;
  return now;
}

// The first n bytes of a block (a multiple of 16) get the new scale; thread i of all, four loads in flight.
template <int MODE>
__device__ __forceinline__ void rescale(uint8_t* block, int n, float was, float rcp, int i, int all) {
  uint4* at = reinterpret_cast<uint4*>(block);
  n /= 16;
  for (int c0 = i; c0 < n; c0 += 4 * all) {
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k * all < n) u[k] = at[c0 + k * all];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c0 + k * all >= n) break;
      uint32_t* w = reinterpret_cast<uint32_t*>(&u[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = qdq_code4_values<MODE>(w[j]);
        w[j] = kv8_code4<MODE>(__fmul_rn(x.x, was), __fmul_rn(x.y, was), __fmul_rn(x.z, was), __fmul_rn(x.w, was), rcp);
      }
      at[c0 + k * all] = u[k];
    }
  }
}

// A CTA takes the tokens of a row that fall on one page, and some of the heads: first K and V
// blocks, which have a scale to agree on, then query heads.  The next block's loads are in
// flight while one is worked on.
template <int MODE, int DIM, int NT, int U>
__global__ void __launch_bounds__(NT) kv8_rotary_kernel(const __grid_constant__ RotaryParams a, int blocks, int per) {
  constexpr int UN = DIM / 16;  // units of a head
  __shared__ float red[2][NT / 32];
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x;
  if (p.cu && blockIdx.y == 0)
    kv8_fill<DIM>(p, (int64_t)blockIdx.x * (NT / 32) + tid / 32, (int64_t)gridDim.x * (NT / 32), tid % 32);
  const int64_t r = blockIdx.x / blocks;
  int64_t base;
  int n;
  const bool whole = kv8_row(p, r, base, n);  // queries of other rows are kv8_fill's
  const int64_t st = p.lengths[r], b = (st >> p.shift) + blockIdx.x % blocks;
  const int64_t lo = st > b * p.page ? st : b * p.page;
  const int64_t hi = st + n < (b + 1) * p.page ? st + n : (b + 1) * p.page;
  if (lo >= hi) return;
  const int64_t id = st >= 0 && b < p.cols ? p.table[r * p.cols + b] : -1;
  const bool paged = id >= 0 && id < p.pages;
  const int count = (int)(hi - lo) * UN, old = (int)(lo - b * p.page), kv = 2 * p.heads;
  const int first = blockIdx.y * per, last = min(first + per, kv + p.heads * p.group);

  float c[U][8], s[U][8];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int at = tid + j * NT;
    if (at < count && unit_of(a, at % UN).turns) angles(a, lo + at / UN, at % UN, c[j], s[j]);
  }
  // block i: K and V of head i / 2 in turn, then the query heads
  auto wanted = [&](int i) { return i < kv ? paged : whole; };
  auto tile_of = [&](int i) { return ((i & 1) * p.pages + id) * p.heads + i / 2; };
  auto load = [&](int i, uint4 (&u)[U][2], float& was) {
    const __nv_bfloat16* x;
    int64_t row, token;
    if (i >= kv) x = a.q + (i - kv) * a.q_head, row = a.q_row, token = a.q_token;
    else if (i & 1) x = p.v + (i / 2) * p.v_head, row = p.v_row, token = p.v_token;
    else x = p.x + (i / 2) * p.x_head, row = p.x_row, token = p.x_token;
    x += kv8_at(p, r, base, lo - st, row, token);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int at = tid + j * NT;
      const Unit w = unit_of(a, at % UN);
      u[j][0] = u[j][1] = make_uint4(0, 0, 0, 0);
      if (at < count) {
        u[j][0] = __ldg(reinterpret_cast<const uint4*>(x + (at / UN) * token + 8 * w.c0));
        u[j][1] = __ldg(reinterpret_cast<const uint4*>(x + (at / UN) * token + 8 * w.c1));
      }
    }
    was = i < kv && old > 0 ? p.scales[tile_of(i)] : 0.f;
  };
  uint4 next[U][2];
  float next_was = 0.f;
  if (wanted(first)) load(first, next, next_was);
  for (int i = first; i < last; ++i) {
    float x[U][2][8];
#pragma unroll
    for (int j = 0; j < U; ++j) bf16x8(next[j][0], x[j][0]), bf16x8(next[j][1], x[j][1]);
    const float was = next_was;
    if (i + 1 < last && wanted(i + 1)) load(i + 1, next, next_was);
    if (!wanted(i)) continue;
    if (i >= kv || !(i & 1)) {
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (unit_of(a, (tid + j * NT) % UN).turns && tid + j * NT < count) turn16(x[j][0], x[j][1], c[j], s[j], a.inter);
    }
    if (i >= kv) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int at = tid + j * NT;
        if (at < count) {
          const Unit w = unit_of(a, at % UN);
          __nv_bfloat16* o = p.o + ((base + lo - st + at / UN) * (p.heads * p.group) + i - kv) * DIM;
          *reinterpret_cast<uint4*>(o + 8 * w.c0) = bf16x8_of(x[j][0]);
          *reinterpret_cast<uint4*>(o + 8 * w.c1) = bf16x8_of(x[j][1]);
        }
      }
      continue;
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) m = most16(x[j][0], x[j][1], m);
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
    float rcp;
    const float now = block_scale<MODE>(was, m, rcp);
    const int64_t tile = tile_of(i);
    uint8_t* out = p.codes + tile * p.page * DIM;
    if (now > was) rescale<MODE>(out, old * DIM, was, rcp, tid, NT);
    if (tid == 0 && (now != was || old == 0)) p.scales[tile] = now;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int at = tid + j * NT;
      if (at < count) {
        const Unit w = unit_of(a, at % UN);
        uint8_t* to = out + (old + at / UN) * DIM;
        *reinterpret_cast<uint2*>(to + 8 * w.c0) = code8<MODE>(x[j][0], rcp);
        *reinterpret_cast<uint2*>(to + 8 * w.c1) = code8<MODE>(x[j][1], rcp);
      }
    }
  }
}

// One token per row: DIM / 16 lanes take a head of it, so a warp 4 (or 8) heads.  (64 rows x 48 heads 2.7 us.)
template <int MODE, int DIM>
__global__ void __launch_bounds__(128) kv8_rotary_one_kernel(const __grid_constant__ RotaryParams a, int groups) {
  constexpr int UN = DIM / 16, G = 32 / UN;
  const Kv8Params& p = a.p;
  const int lane = threadIdx.x % 32, u = lane % UN;
  const int64_t warp = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  if (p.cu) kv8_fill<DIM>(p, warp, (int64_t)gridDim.x * 4, lane);
  const int64_t r = warp / groups;
  if (r >= p.rows) return;
  int64_t base;
  int n;
  const bool whole = kv8_row(p, r, base, n);
  if (n == 0) return;
  const int64_t st = p.lengths[r], b = st >> p.shift;
  const int64_t id = st >= 0 && b < p.cols ? p.table[r * p.cols + b] : -1;
  const int old = (int)(st & (p.page - 1)), kv = 2 * p.heads;
  const int i = (int)(warp % groups) * G + lane / UN;
  const bool is_q = i >= kv, have = is_q ? whole && i < kv + p.heads * p.group : id >= 0 && id < p.pages;
  const Unit w = unit_of(a, u);
  const int64_t tile = ((i & 1) * p.pages + id) * p.heads + i / 2;
  float x[2][8], was = 0.f, m = 0.f;
  if (have) {
    const __nv_bfloat16* from =
        is_q ? a.q + kv8_at(p, r, base, 0, a.q_row, a.q_token) + (i - kv) * a.q_head
             : i & 1 ? p.v + kv8_at(p, r, base, 0, p.v_row, p.v_token) + (i / 2) * p.v_head
                     : p.x + kv8_at(p, r, base, 0, p.x_row, p.x_token) + (i / 2) * p.x_head;
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(from + 8 * w.c0));
    const uint4 hi = __ldg(reinterpret_cast<const uint4*>(from + 8 * w.c1));
    if (!is_q && old > 0) was = p.scales[tile];
    float c[8], s[8];
    const bool turns = w.turns && (is_q || !(i & 1));
    if (turns) angles(a, st, u, c, s);
    bf16x8(lo, x[0]), bf16x8(hi, x[1]);
    if (turns) turn16(x[0], x[1], c, s, a.inter);
    m = most16(x[0], x[1], 0.f);
  }
#pragma unroll
  for (int d = 1; d < UN; d <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  float rcp;
  const float now = block_scale<MODE>(was, m, rcp);
  __syncwarp();  // every lane has read the block's scale
  unsigned grown = __ballot_sync(0xffffffffu, have && !is_q && old > 0 && now > was && u == 0);
  for (; grown; grown &= grown - 1) {  // the whole warp writes a block's old codes again
    const int from = __ffs(grown) - 1;
    rescale<MODE>(p.codes + __shfl_sync(0xffffffffu, tile, from) * p.page * DIM, old * DIM,
                  __shfl_sync(0xffffffffu, was, from), __shfl_sync(0xffffffffu, rcp, from), lane, 32);
  }
  if (!have) return;
  if (is_q) {
    __nv_bfloat16* o = p.o + (base * (p.heads * p.group) + i - kv) * DIM;
    *reinterpret_cast<uint4*>(o + 8 * w.c0) = bf16x8_of(x[0]);
    *reinterpret_cast<uint4*>(o + 8 * w.c1) = bf16x8_of(x[1]);
  } else {
    if (u == 0 && (now != was || old == 0)) p.scales[tile] = now;
    uint8_t* to = p.codes + (tile * p.page + old) * DIM;
    *reinterpret_cast<uint2*>(to + 8 * w.c0) = code8<MODE>(x[0], rcp);
    *reinterpret_cast<uint2*>(to + 8 * w.c1) = code8<MODE>(x[1], rcp);
  }
}

template <int MODE, int DIM>
gdn_status run(const RotaryParams& a, cudaStream_t st) {
  const Kv8Params& p = a.p;
  const int64_t heads = 2 * (int64_t)p.heads + (int64_t)p.heads * p.group;
  if (p.tokens == 1) {
    constexpr int G = 32 / (DIM / 16);
    const int64_t groups = (heads + G - 1) / G, ctas = (p.rows * groups + 3) / 4;
    if (ctas > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
    kv8_rotary_one_kernel<MODE, DIM><<<(unsigned)ctas, 128, 0, st>>>(a, (int)groups);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  }
  // pages that n consecutive positions can touch
  const int blocks = (p.tokens + p.page - 2) / p.page + 1;
  if (p.rows * blocks > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
  // heads per CTA, whose loads overlap and which share the angles: up to 8 while 152 SMs still get eight
  // CTAs each (8 prompts to 4096 tokens: four 95.5 us, eight 88.7, sixteen 92.5)
  int per = 1;
  while (per < 8 && per < heads && p.rows * blocks * heads / (2 * per) >= 152 * 8) per *= 2;
  const int64_t runs = (heads + per - 1) / per;
  if (runs > 65535) return GDN_ERR_UNSUPPORTED_SHAPE;
  const dim3 grid((unsigned)(p.rows * blocks), (unsigned)runs);
  const int units = (p.tokens < p.page ? p.tokens : p.page) * (DIM / 16);
  if (units <= 32) kv8_rotary_kernel<MODE, DIM, 32, 1><<<grid, 32, 0, st>>>(a, blocks, per);
  else if (units <= 128) kv8_rotary_kernel<MODE, DIM, 128, 1><<<grid, 128, 0, st>>>(a, blocks, per);
  else if (units <= 256) kv8_rotary_kernel<MODE, DIM, 128, 2><<<grid, 128, 0, st>>>(a, blocks, per);
  else if (units <= 512) kv8_rotary_kernel<MODE, DIM, 256, 2><<<grid, 256, 0, st>>>(a, blocks, per);
  else kv8_rotary_kernel<MODE, DIM, 512, 2><<<grid, 512, 0, st>>>(a, blocks, per);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

gdn_status launch_kv8_rotary(const Kv8Params& p, const Kv8Rotary& w, int mode, int dim, cudaStream_t st) {
  RotaryParams a;
  a.p = p;
  a.q = w.q, a.cos = w.cos, a.sin = w.sin, a.positions = w.positions;
  a.q_row = w.q_row, a.q_token = w.q_token, a.q_head = w.q_head;
  a.half = w.dim / 2, a.inter = w.interleaved;
  if (mode == GDN_QDQ_E4M3) return dim == 128 ? run<GDN_QDQ_E4M3, 128>(a, st) : run<GDN_QDQ_E4M3, 64>(a, st);
  return dim == 128 ? run<GDN_QDQ_INT8, 128>(a, st) : run<GDN_QDQ_INT8, 64>(a, st);
}

}  // namespace gdn
