// Attention of few query rows over the 8-bit paged cache: the queries of a row
// times the query heads of a K/V head are at most 16, so one 16-row tile of
// warp-level products holds them all and every code is read once.  The bytes of
// the codes bound it.
//
// Work.  The keys of one (row, K/V head), a segment, are cut into tiles of 32.  All
// tiles of all segments form one line, of which every warp takes an equal,
// contiguous share, so uneven lengths and a single long row fill the GPU alike.
// A warp that holds a whole segment writes its output; otherwise it has a part
// (its output normalised over its own keys, and their log-sum-exp), the parts of
// one CTA are joined in shared memory, and what is left goes to the workspace,
// where a second launch joins the parts of a segment in order.  Short tables
// give one CTA per segment instead, and then nothing is left to join.
//
// A warp runs by itself: a ring of S tiles (K and V, by TMA, 128- or 64-byte
// swizzle) that its lane 0 refills, products m16n8k16 in fp16 with fp32 sums (the
// codes are exact in fp16; q keeps its bits by a power of two per row), and an
// online softmax.  A block's V scale multiplies the probabilities, so these run
// against a second maximum, of score + log2(scale), and stay within [0, 1] for
// any scales.
#include <cuda.h>

#include "kv8.cuh"
#include "launch.h"

namespace gdn {

namespace {

__device__ int g_kv8_device_error;

constexpr int kTile = 32, kWarps = 8;
constexpr int kSegmentTiles = 64;  // tables up to this many tiles: one CTA per segment

struct DecodeArgs {
  Kv8Params p;
  CUtensorMap map;
  float* ws;
  int whole;  // one CTA per segment
};

template <int DIM>
constexpr int kSlot = 16 * DIM + 16;  // a part: outputs of 16 rows, their log2-sum-exp2

__device__ __forceinline__ int tiles_of(const Kv8Span& s) {
  return s.end > s.begin ? (s.end + kTile - 1) / kTile - s.begin / kTile : 0;
}

// Shares of the line of tiles: CTA c of n, warp w of it.
__device__ __forceinline__ int64_t cta_start(int64_t all, int64_t c, int64_t n) {
  return all / n * c + all % n * c / n;
}
__device__ __forceinline__ int64_t warp_start(int64_t lo, int64_t hi, int w) {
  return lo + (hi - lo) * w / kWarps;
}
// CTAs that take part: at least one tile for each of their warps
__device__ __forceinline__ int64_t ctas_for(int64_t all, int64_t grid) {
  const int64_t n = (all + kWarps - 1) / kWarps;
  return n < 1 ? 1 : n < grid ? n : grid;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Tiles per K/V head of rows [0, r1).
__device__ __forceinline__ int64_t tiles_before(const Kv8Params& p, int64_t r1, int lane) {
  int64_t t = 0;
  for (int64_t r = lane; r < r1; r += 32) t += tiles_of(kv8_span(p, r));
  return warp_sum64(t);
}

// The tile at place u of the line: its segment, and where that begins.
struct Cursor {
  int64_t r;      // row
  int h;          // K/V head
  int tile;       // tile of the row, counted from key 0
  int t0, t1;     // the segment's tiles
  int64_t u0;     // the segment's first place
};

__device__ __forceinline__ Cursor locate(const Kv8Params& p, int64_t u, int lane) {
  Cursor c;
  int64_t before = 0;
  for (int64_t r0 = 0;; r0 += 32) {
    const int64_t r = r0 + lane;
    const int64_t mine = r < p.rows ? tiles_of(kv8_span(p, r)) : 0;
    int64_t x = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, (before + x) * p.heads > u);
    if (hit || r0 + 32 >= p.rows) {
      const int at = hit ? __ffs(hit) - 1 : 31;
      c.r = r0 + at;
      c.u0 = (before + __shfl_sync(0xffffffffu, x - mine, at)) * p.heads;
      break;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  const Kv8Span s = kv8_span(p, c.r < p.rows ? c.r : p.rows - 1);
  c.t0 = s.begin / kTile;
  c.t1 = c.t0 + tiles_of(s);
  const int64_t n = c.t1 - c.t0, off = u - c.u0;
  c.h = n > 0 ? (int)(off / n) : 0;
  c.u0 += c.h * n;
  c.tile = c.t0 + (n > 0 ? (int)(off % n) : 0);
  return c;
}

// To the first tile of the next segment.
__device__ __forceinline__ void next_segment(const Kv8Params& p, Cursor& c) {
  c.u0 += c.t1 - c.t0;
  if (++c.h == p.heads) {
    c.h = 0;
    int n = 0;
    while (++c.r < p.rows) {
      const Kv8Span s = kv8_span(p, c.r);
      c.t0 = s.begin / kTile;
      n = tiles_of(s);
      if (n) break;
    }
    c.t1 = c.t0 + n;
  }
  c.tile = c.t0;
}

// Output rows of a segment: row i of the tile is query i / group, head i % group.
template <int DIM>
__device__ __forceinline__ int64_t out_row(const Kv8Params& p, const Kv8Span& s, int h, int i) {
  return (s.base + i / p.group) * (p.heads * p.group) + h * p.group + i % p.group;
}

template <int MODE, int DIM, int S>
__global__ void __launch_bounds__(kWarps * 32, 1)
    kv8_decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int KSTEPS = DIM / 16, NT = DIM / 8;      // 16-byte chunks of a row; n tiles of V
  constexpr int kBytes = kTile * DIM;                 // K or V of a tile
  constexpr int kRowMask = DIM == 128 ? 7 : 3, kRowShift = DIM == 128 ? 0 : 1;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[kWarps][S];
  __shared__ float4 meta[kWarps][S];   // per half tile: K scale, log2 of V scale
  __shared__ int valid[kWarps][S];     // bit i: half i has a page
  __shared__ int64_t s_u0[kWarps];     // segment of a warp's part, -1: none
  __shared__ float s_lse[kWarps][16];
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, t = lane % 4;
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* ring = smem + warp * (S * 2 * kBytes);

  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&bars[warp][i], 1);
    fence_mbar_init();
  }
  __syncwarp();

  // ---- this warp's share ----
  int64_t lo, hi;
  Cursor pc;
  if (a.whole) {
    pc.r = blockIdx.x / p.heads, pc.h = blockIdx.x % p.heads, pc.u0 = 0;
    const Kv8Span s = kv8_span(p, pc.r);
    pc.t0 = s.begin / kTile, pc.t1 = pc.t0 + tiles_of(s);
    const int n = pc.t1 - pc.t0;
    lo = warp_start(0, n, warp), hi = warp_start(0, n, warp + 1);
    pc.tile = pc.t0 + (int)lo;
    if (n == 0) lo = hi = 0;
  } else {
    const int64_t all = tiles_before(p, p.rows, lane) * p.heads;
    const int64_t n = ctas_for(all, gridDim.x);
    lo = hi = 0;
    if (blockIdx.x < n && all > 0) {
      const int64_t c0 = cta_start(all, blockIdx.x, n), c1 = cta_start(all, blockIdx.x + 1, n);
      lo = warp_start(c0, c1, warp), hi = warp_start(c0, c1, warp + 1);
      if (lo < hi) pc = locate(p, lo, lane);
    }
  }
  // rows that see nothing at all: zeros, written by some warp
  for (int64_t r = (int64_t)blockIdx.x * kWarps + warp; r < p.rows; r += (int64_t)gridDim.x * kWarps) {
    const Kv8Span s = kv8_span(p, r);
    if (s.n == 0 || tiles_of(s) > 0) continue;
    const int64_t rows = (int64_t)s.n * p.heads * p.group, o0 = s.base * p.heads * p.group;
    for (int64_t i = lane; i < rows * (DIM / 8); i += 32)
      reinterpret_cast<uint4*>(p.o + o0 * DIM)[i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int64_t i = lane; i < rows; i += 32) p.lse[o0 + i] = -INFINITY;
  }

  // ---- loads: the pages and scales of 32 blocks ahead lie in the lanes ----
  int w_id = -1, w_base = 0, w_h = -1;
  int64_t w_r = -1;
  float w_ks = 0.f, w_lv = -INFINITY;
  const int two = p.page < kTile;  // two pages per tile
  auto issue = [&](int st) {
    const int j0 = pc.tile * kTile, first = j0 >> p.shift;
    if (pc.r != w_r || pc.h != w_h || first >= w_base + 32 || first < w_base) {
      w_r = pc.r, w_h = pc.h, w_base = first;
      const int at = first + lane;
      w_id = at < p.cols && (int64_t)at * p.page < (int64_t)pc.t1 * kTile
                 ? p.table[w_r * p.cols + at] : -1;
      w_ks = 0.f, w_lv = -INFINITY;
      if (w_id < 0 || w_id >= p.pages) {
        w_id = -1;
      } else {
        const int64_t tile = (int64_t)w_id * p.heads + w_h;
        w_ks = p.scales[tile];
        w_lv = lg2_approx(p.scales[tile + p.pages * p.heads]);
      }
    }
    const int from = first - w_base;
    const int id0 = __shfl_sync(0xffffffffu, w_id, from);
    const float ks0 = __shfl_sync(0xffffffffu, w_ks, from), lv0 = __shfl_sync(0xffffffffu, w_lv, from);
    const int id1 = __shfl_sync(0xffffffffu, w_id, from + two);
    const float ks1 = __shfl_sync(0xffffffffu, w_ks, from + two);
    const float lv1 = __shfl_sync(0xffffffffu, w_lv, from + two);
    if (lane == 0) {
      meta[warp][st] = make_float4(ks0, lv0, ks1, lv1);
      valid[warp][st] = (id0 >= 0) | (id1 >= 0) << 1;
      unsigned char* k = ring + st * 2 * kBytes;
      const int per = two ? kBytes / 2 : kBytes;
      mbar_expect_tx(&bars[warp][st],
                     (uint32_t)(per * 2 * ((id0 >= 0) + (two && id1 >= 0))));
      if (id0 >= 0) {
        const int z = id0 * p.heads + pc.h, y = j0 & (p.page - 1);
        tma_load_3d(k, &a.map, 0, y, z, &bars[warp][st]);
        tma_load_3d(k + kBytes, &a.map, 0, y, z + (int)(p.pages * p.heads), &bars[warp][st]);
      }
      if (two && id1 >= 0) {
        const int z = id1 * p.heads + pc.h;
        tma_load_3d(k + kBytes / 2, &a.map, 0, 0, z, &bars[warp][st]);
        tma_load_3d(k + kBytes + kBytes / 2, &a.map, 0, 0, z + (int)(p.pages * p.heads),
                    &bars[warp][st]);
      }
    }
    if (++pc.tile == pc.t1) next_segment(p, pc);
  };

  int64_t issued = lo;
  Cursor cc = pc;  // the consumer's place
  for (int i = 0; i < S && issued < hi; ++i, ++issued) issue(i);

  // ---- segments ----
  bool bad = false;
  int st = 0;
  uint32_t parity = 0;
  float oacc[NT][4];
  float lsum[2], m[2], mv[2];
  Kv8Span sp;
  int64_t part = -1;  // segment left in registers at the end
  int64_t u_done = lo;
  for (int64_t u = lo; u < hi && !bad;) {
    const int64_t u0 = cc.u0, u1 = u0 + (cc.t1 - cc.t0);
    const int64_t stop = u1 < hi ? u1 : hi;
    sp = kv8_span(p, cc.r);
    const int rows = sp.n * p.group;
    // q fragments: rows g and g + 8, element pairs in the order kv8_half2 gives K's
    uint32_t qf[KSTEPS][4];
    float rowfac[2];
    int beg[2], end[2];
    {
      uint2 raw[2][KSTEPS];
      float most[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = g + 8 * e;
        const int qi = i / p.group;
        const bool have = i < rows;
        if (have) kv8_seen(p, sp, qi, beg[e], end[e]); else beg[e] = end[e] = 0;
        const __nv_bfloat16* x = p.x + kv8_at(p, cc.r, sp.base, qi, p.x_row, p.x_token) +
                                 (cc.h * p.group + i % p.group) * p.x_head + 4 * t;
#pragma unroll
        for (int c = 0; c < KSTEPS; ++c) {
          raw[e][c] = have ? *reinterpret_cast<const uint2*>(x + 16 * c) : make_uint2(0, 0);
          float f[4];
          bf16x4(raw[e][c], f);
          most[e] = fmaxf(most[e], fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
        }
        most[e] = fmaxf(most[e], __shfl_xor_sync(0xffffffffu, most[e], 1));
        most[e] = fmaxf(most[e], __shfl_xor_sync(0xffffffffu, most[e], 2));
        float to, back;
        kv8_q_factor(most[e], to, back);
        rowfac[e] = back * p.scale * kLog2eF * (MODE == GDN_QDQ_E4M3 ? 256.f : 1.f);
#pragma unroll
        for (int c = 0; c < KSTEPS; ++c) {
          float f[4];
          bf16x4(raw[e][c], f);
          qf[c][e] = pack_f16(f[0] * to, f[2] * to);
          qf[c][2 + e] = pack_f16(f[1] * to, f[3] * to);
        }
      }
    }
    // tiles inside [in0, in1) need no mask
    int in0, in1;
    {
      int b0, e0, b1, e1;
      kv8_seen(p, sp, 0, b0, e0);
      kv8_seen(p, sp, sp.n - 1, b1, e1);
      in0 = b1, in1 = e0;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;
    lsum[0] = lsum[1] = 0.f;
    m[0] = m[1] = mv[0] = mv[1] = -INFINITY;

    for (; u < stop; ++u, ++cc.tile) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[warp][st], parity))) {
        bad = true;
        break;
      }
      const unsigned char* kt = ring + st * 2 * kBytes;
      const uint32_t kaddr = smem_u32(kt), vaddr = kaddr + kBytes;
      const float4 sc = meta[warp][st];
      const int have = valid[warp][st];
      // ---- scores: n tile j = keys 8 j .. 8 j + 7 ----
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        const int row = 8 * j + lane % 8;
#pragma unroll
        for (int q = 0; q < KSTEPS / 4; ++q) {
          uint32_t r[4];
          ldsm_x4(r, kaddr + row * DIM + (((4 * q + lane / 8) ^ ((row >> kRowShift) & kRowMask)) << 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            kv8_half2<MODE>(r[i], b0, b1);
            mma_f16(s[j], qf[4 * q + i], b0, b1);
          }
        }
      }
      const int j0 = cc.tile * kTile;
      const bool mask = have != 3 || j0 < in0 || j0 + kTile > in1;
      float half[2][2];  // row, half tile: largest score
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float fac = rowfac[e] * (f ? sc.z : sc.x);
          float top = -INFINITY;
#pragma unroll
          for (int j = 2 * f; j < 2 * f + 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = s[j][2 * e + i] * fac;
              if (mask) {
                const int at = j0 + 8 * j + 2 * t + i;
                if (at < beg[e] || at >= end[e] || !(have >> f & 1)) x = -INFINITY;
              }
              s[j][2 * e + i] = x;
              top = fmaxf(top, x);
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          half[e][f] = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        }
      }
      float f_half[2][2], scale_o[2];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float nm = fmaxf(m[e], fmaxf(half[e][0], half[e][1]));
        const float nv = fmaxf(mv[e], fmaxf(half[e][0] + sc.y, half[e][1] + sc.w));
        const float um = nm == -INFINITY ? 0.f : nm, uv = nv == -INFINITY ? 0.f : nv;
        lsum[e] *= ex2_approx_f(m[e] - um);
        scale_o[e] = ex2_approx_f(mv[e] - uv);
        moved |= nv != mv[e];
        f_half[e][0] = ex2_approx_f(fminf(um + sc.y - uv, 126.f));
        f_half[e][1] = ex2_approx_f(fminf(um + sc.w - uv, 126.f));
        m[e] = nm, mv[e] = nv;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w = ex2_approx_f(s[j][2 * e + i] - um);
            lsum[e] += w;
            s[j][2 * e + i] = w * f_half[e][j / 2];
          }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          oacc[i][0] *= scale_o[0], oacc[i][1] *= scale_o[0];
          oacc[i][2] *= scale_o[1], oacc[i][3] *= scale_o[1];
        }
      }
      // ---- output: 16 keys per step; a 16-byte chunk of V gives two n tiles ----
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t pf[4];
        pf[0] = pack_f16(s[2 * k][0], s[2 * k][1]);
        pf[1] = pack_f16(s[2 * k][2], s[2 * k][3]);
        pf[2] = pack_f16(s[2 * k + 1][0], s[2 * k + 1][1]);
        pf[3] = pack_f16(s[2 * k + 1][2], s[2 * k + 1][3]);
        const int row = 16 * k + (lane / 8 & 1) * 8 + lane % 8;
#pragma unroll
        for (int c = 0; c < KSTEPS; c += 2) {
          uint32_t r[4];
          ldsm_x4_t(r, vaddr + row * DIM + (((c + lane / 16) ^ ((row >> kRowShift) & kRowMask)) << 4));
          uint32_t e0, o0, e1, o1;
          kv8_half2<MODE>(r[0], e0, o0);
          kv8_half2<MODE>(r[1], e1, o1);
          mma_f16(oacc[2 * c], pf, e0, e1);
          mma_f16(oacc[2 * c + 1], pf, o0, o1);
          kv8_half2<MODE>(r[2], e0, o0);
          kv8_half2<MODE>(r[3], e1, o1);
          mma_f16(oacc[2 * c + 2], pf, e0, e1);
          mma_f16(oacc[2 * c + 3], pf, o0, o1);
        }
      }
      __syncwarp();  // the tile has been read by every lane
      if (issued < hi) {
        issue(st);
        ++issued;
      }
      if (++st == S) st = 0, parity ^= 1;
    }
    u_done = u;
    if (bad) break;

    // ---- the segment's output over this warp's keys ----
    float lse2[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = lsum[e];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      lse2[e] = l > 0.f ? m[e] + log2f(l) : -INFINITY;
      // mv is -inf where every V scale seen is 0
      const float fac = l > 0.f && mv[e] > -INFINITY
                            ? ex2_approx_f(mv[e] - m[e] + kKv8Shift<MODE>) / l : 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) oacc[i][2 * e] *= fac, oacc[i][2 * e + 1] *= fac;
    }
    const bool whole = lo <= u0 && u1 <= hi;
    if (whole || u1 < hi) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = g + 8 * e;
        if (i >= rows) continue;
        if (whole) {
          const int64_t at = out_row<DIM>(p, sp, cc.h, i);
          __nv_bfloat16* o = p.o + at * DIM + 4 * t;
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c)
            *reinterpret_cast<uint2*>(o + 16 * c) =
                make_uint2(pack_bf16(oacc[2 * c][2 * e], oacc[2 * c + 1][2 * e]),
                           pack_bf16(oacc[2 * c][2 * e + 1], oacc[2 * c + 1][2 * e + 1]));
          if (p.lse && t == 0) p.lse[at] = lse2[e] * 0.6931471805599453f;
        } else {
          // began in an earlier warp, ends here: to the workspace
          float* o = a.ws + ((int64_t)blockIdx.x * kWarps + warp) * 2 * kSlot<DIM>;
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c)
            *reinterpret_cast<float4*>(o + i * DIM + 16 * c + 4 * t) =
                make_float4(oacc[2 * c][2 * e], oacc[2 * c + 1][2 * e], oacc[2 * c][2 * e + 1],
                            oacc[2 * c + 1][2 * e + 1]);
          if (t == 0) o[16 * DIM + i] = lse2[e];
        }
      }
    } else {
      part = u0;
      if (t == 0) s_lse[warp][g] = lse2[0], s_lse[warp][g + 8] = lse2[1];
    }
    if (u < hi) {
      // the next segment; cc.tile stands at its end
      cc.tile = cc.t1;
      next_segment(p, cc);
    }
  }
  if (bad) {
    // the copies in flight, from tile u on, land within the bounded waits
    for (int64_t i = u_done; i < issued && lane == 0; ++i) {
      mbar_wait(&bars[warp][st], parity);
      if (++st == S) st = 0, parity ^= 1;
    }
    if (lane == 0) atomicOr(&g_kv8_device_error, 1);
    part = -1;
  }

  // ---- parts of one CTA ----
  if (lane == 0) s_u0[warp] = part;
  __syncthreads();  // every ring is done with
  float* parts = reinterpret_cast<float*>(smem);  // [warp][16][DIM]
  if (part >= 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float* o = parts + (warp * 16 + g + 8 * e) * DIM + 4 * t;
#pragma unroll
      for (int c = 0; c < KSTEPS; ++c)
        *reinterpret_cast<float4*>(o + 16 * c) =
            make_float4(oacc[2 * c][2 * e], oacc[2 * c + 1][2 * e], oacc[2 * c][2 * e + 1],
                        oacc[2 * c + 1][2 * e + 1]);
    }
  }
  __syncthreads();
  // a warp whose part is the first of its segment here knows the segment's place
  __shared__ int64_t s_u1[kWarps], s_base[kWarps], s_hi[kWarps], s_lo[kWarps];
  __shared__ int s_rows[kWarps], s_h[kWarps];
  if (lane == 0 && part >= 0) {
    s_u1[warp] = cc.u0 + (cc.t1 - cc.t0), s_base[warp] = sp.base, s_rows[warp] = sp.n * p.group;
    s_h[warp] = cc.h, s_hi[warp] = hi, s_lo[warp] = lo;
  }
  __syncthreads();
  for (int w0 = 0; w0 < kWarps;) {
    const int64_t u0 = s_u0[w0];
    if (u0 < 0) {
      ++w0;
      continue;
    }
    int w1 = w0 + 1, last = w0;
    // empty shares lie between the warps of one segment
    for (; w1 < kWarps && (s_u0[w1] == u0 || s_u0[w1] < 0); ++w1)
      if (s_u0[w1] == u0) last = w1;
    const bool whole = s_lo[w0] <= u0 && s_hi[last] >= s_u1[w0];
    const int rows = s_rows[w0];
    Kv8Span f;
    f.base = s_base[w0];
    float* slot = a.ws + (((int64_t)blockIdx.x * kWarps + w0) * 2 + 1) * kSlot<DIM>;
    for (int at = tid; at < rows * (DIM / 4); at += kWarps * 32) {
      const int i = at / (DIM / 4), d = at % (DIM / 4) * 4;
      float top = -INFINITY;
      for (int w = w0; w <= last; ++w)
        if (s_u0[w] == u0) top = fmaxf(top, s_lse[w][i]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
      if (top > -INFINITY) {
        for (int w = w0; w <= last; ++w) {
          if (s_u0[w] != u0) continue;
          const float c = ex2_approx_f(s_lse[w][i] - top);
          const float4 x = *reinterpret_cast<const float4*>(parts + (w * 16 + i) * DIM + d);
          l += c;
          o.x = fmaf(c, x.x, o.x), o.y = fmaf(c, x.y, o.y);
          o.z = fmaf(c, x.z, o.z), o.w = fmaf(c, x.w, o.w);
        }
        const float inv = 1.f / l;
        o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
      }
      const float lse2 = top > -INFINITY ? top + log2f(l) : -INFINITY;
      if (whole) {
        const int64_t to = out_row<DIM>(p, f, s_h[w0], i);
        *reinterpret_cast<uint2*>(p.o + to * DIM + d) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
        if (p.lse && d == 0) p.lse[to] = lse2 * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(slot + i * DIM + d) = o;
        if (d == 0) slot[16 * DIM + i] = lse2;
      }
    }
    w0 = w1;
  }
}

// Joins the parts of a segment that several CTAs hold: one CTA per (segment,
// output row), its warps over the parts, their sums in warp order.
template <int DIM>
__global__ void __launch_bounds__(256) kv8_join_kernel(const __grid_constant__ DecodeArgs a, int grid) {
  constexpr int kList = 1024;
  __shared__ float s_w[kList];
  __shared__ int s_at[kList];
  __shared__ float red[8];
  __shared__ __align__(16) float s_o[8][DIM];
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t r = blockIdx.x / p.heads;
  const int h = blockIdx.x % p.heads, i = blockIdx.y;
  const Kv8Span sp = kv8_span(p, r);
  const int n = tiles_of(sp);
  if (n == 0 || i >= sp.n * p.group) return;
  __shared__ int64_t s_all, s_before;
  if (warp == 0) {
    const int64_t all = tiles_before(p, p.rows, lane), before = tiles_before(p, r, lane);
    if (lane == 0) s_all = all * p.heads, s_before = before * p.heads;
  }
  __syncthreads();
  const int64_t all = s_all, ctas = ctas_for(all, grid);
  const int64_t u0 = s_before + (int64_t)h * n, u1 = u0 + n;
  // CTAs whose shares meet the segment: c with start(c) < u1 and start(c + 1) > u0
  int64_t c0 = u0 * ctas / all, c1;
  while (c0 > 0 && cta_start(all, c0, ctas) > u0) --c0;
  while (cta_start(all, c0 + 1, ctas) <= u0) ++c0;
  c1 = (u1 - 1) * ctas / all;
  while (c1 > 0 && cta_start(all, c1, ctas) > u1 - 1) --c1;
  while (cta_start(all, c1 + 1, ctas) <= u1 - 1) ++c1;
  // one entry per CTA for what its warps left of the segment, and one for a warp
  // that goes on after the segment's end
  const int entries = (int)(c1 - c0 + 1) + 1;
  if (entries > kList) return;
  float top = -INFINITY;
  bool direct = false;
  for (int k = tid; k < entries; k += 256) {
    const int64_t c = k < entries - 1 ? c0 + k : c1;
    const int64_t lo = cta_start(all, c, ctas), hi = cta_start(all, c + 1, ctas);
    int at = -1;
    int64_t first = -1, last_hi = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int64_t s = warp_start(lo, hi, w), e = warp_start(lo, hi, w + 1);
      if (s >= e || s >= u1 || e <= u0) continue;
      if (s <= u0 && e >= u1) {
        direct = true;
      } else if (e <= u1) {
        if (first < 0) first = s, at = k < entries - 1 ? (int)((c * kWarps + w) * 2 + 1) : at;
        last_hi = e;
      } else if (k == entries - 1) {
        at = (int)((c * kWarps + w) * 2);
      }
    }
    if (first >= 0 && first <= u0 && last_hi >= u1) direct = true;
    s_at[k] = at;
    const float x = at >= 0 && !direct ? a.ws[(int64_t)at * kSlot<DIM> + 16 * DIM + i] : -INFINITY;
    s_w[k] = x;
    top = fmaxf(top, x);
  }
  // (the workspace was written by the launch before, which has completed)
  if (__syncthreads_or(direct)) return;  // written already
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  for (int w = 0; w < 8; ++w) top = fmaxf(top, red[w]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  if (top > -INFINITY) {
    for (int k = warp; k < entries; k += 8) {
      if (s_at[k] < 0) continue;
      const float c = ex2_approx_f(s_w[k] - top);
      l += c;
      if (lane < DIM / 4) {
        const float4 x = *reinterpret_cast<const float4*>(a.ws + (int64_t)s_at[k] * kSlot<DIM> + i * DIM + 4 * lane);
        o.x = fmaf(c, x.x, o.x), o.y = fmaf(c, x.y, o.y);
        o.z = fmaf(c, x.z, o.z), o.w = fmaf(c, x.w, o.w);
      }
    }
  }
  __syncthreads();
  if (lane < DIM / 4) *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = o;
  if (lane == 0) red[warp] = l;
  __syncthreads();
  l = 0.f;
  for (int w = 0; w < 8; ++w) l += red[w];
  const int64_t to = out_row<DIM>(p, sp, h, i);
  if (tid < DIM / 2) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < 8; ++w) x += s_o[w][2 * tid], y += s_o[w][2 * tid + 1];
    const float inv = l > 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<uint32_t*>(p.o + to * DIM + 2 * tid) = pack_bf16(x * inv, y * inv);
  }
  if (p.lse && tid == 0) p.lse[to] = l > 0.f ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Most tiles that a row can have, by its table and window.
int64_t most_tiles(const Kv8Params& p) {
  int64_t keys = (int64_t)p.cols * p.page;
  if (p.window > 0 && (int64_t)p.window + p.tokens < keys) keys = (int64_t)p.window + p.tokens;
  return (keys + kTile - 1) / kTile + 1;
}
bool by_segment(const Kv8Params& p) {
  return most_tiles(p) <= kSegmentTiles && p.rows * p.heads <= 0x7fffffffLL;
}
int64_t grid_of(const Kv8Params& p) {
  const int64_t tiles = most_tiles(p) * p.rows * p.heads;
  const int64_t n = (tiles + kWarps - 1) / kWarps;
  return n < 1 ? 1 : n < 152 ? n : 152;
}

template <int MODE, int DIM>
gdn_status run(DecodeArgs& a, cudaStream_t st) {
  constexpr int S = DIM == 128 ? 3 : 6;
  constexpr int bytes = kWarps * S * 2 * kTile * DIM + 1024;
  const Kv8Params& p = a.p;
  const uint32_t box = p.page < kTile ? p.page : kTile;
  a.map = CUtensorMap();
  if (p.pages > 0 && !make_map_3d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, DIM, p.page,
                   (uint64_t)(2 * p.pages * p.heads), DIM, DIM, box,
                   DIM == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return GDN_ERR_CUDA;
  a.whole = by_segment(p);
  const int64_t grid = a.whole ? p.rows * p.heads : grid_of(p);
  auto kern = kv8_decode_kernel<MODE, DIM, S>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return GDN_ERR_CUDA;
  kern<<<(unsigned)grid, kWarps * 32, bytes, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  if (a.whole) return GDN_OK;
  kv8_join_kernel<DIM><<<dim3((unsigned)(p.rows * p.heads), (unsigned)(p.tokens * p.group)), 256, 0, st>>>(a, (int)grid);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

size_t kv8_decode_workspace(const Kv8Params& p, int dim) {
  if (by_segment(p)) return 0;
  return (size_t)grid_of(p) * kWarps * 2 * (16 * dim + 16) * sizeof(float);
}

gdn_status launch_kv8_decode(const Kv8Params& p, int mode, int dim, void* workspace,
                             cudaStream_t st) {
  DecodeArgs a;
  a.p = p;
  a.ws = static_cast<float*>(workspace);
  if (mode == GDN_QDQ_E4M3)
    return dim == 128 ? run<GDN_QDQ_E4M3, 128>(a, st) : run<GDN_QDQ_E4M3, 64>(a, st);
  return dim == 128 ? run<GDN_QDQ_INT8, 128>(a, st) : run<GDN_QDQ_INT8, 64>(a, st);
}

int kv8_device_error(bool reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv8_device_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_kv8_device_error, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  const int u = kv8_prefill_device_error(reset);
  return u < 0 ? -1 : v | u;
}

}  // namespace gdn
