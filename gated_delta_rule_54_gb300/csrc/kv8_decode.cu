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
// where a second launch joins the parts of a segment in order.  Where it is faster
// (by_segment) a CTA has one segment instead, and nothing is left to join.
//
// A warp runs by itself: a ring of S tiles (K and V, by TMA, 128- or 64-byte
// swizzle) that its lane 0 refills, warp products with fp32 sums, and an online
// softmax.  E4M3 scores come from the codes as they are, with q as a sum of two
// 8-bit numbers; INT8 codes, and those of V, are exact in fp16 (q keeps its bits by
// a power of two per row).  A block's V scale multiplies the probabilities, so these run
// against a second maximum, of score + log2(scale), and stay within [0, 1] for
// any scales.
//
// Measured on a GB300 (kernel alone): 64 rows of 2192 .. 8192 keys, 8 K/V heads of
// 128, E4M3, 676 MB: 116 us, 5.8 TB/s (copying: 6.8).  2 rows of 101072 and 131071
// keys, 4 heads, INT8, 260 MB: 55 us.  DRAM is at 72 and 57 %, instruction issue at
// half of its slots from two warps per scheduler; the join takes 8 us.
// The first case with both launches: 12 warps of two tiles (168 registers) took 155 us,
// 8 warps of three 146 (117 without their products), scores from E4M3 codes as they
// are and the leaving out of rows 8-15 made it 126, 32-bit divisions for the shares
// 125 (1024 rows of 16 keys: 81 to 69).
#include <cuda.h>

#include "kv8.cuh"
#include "launch.h"

namespace gdn {

namespace {

__device__ int g_kv8_device_error;

constexpr int kTile = 32, kWarps = 8;

struct DecodeArgs {
  Kv8Params p;
  CUtensorMap map;
  float* ws;        // parts: two slots per warp of the grid
  int64_t* before;  // tiles (of one K/V head) before each row
  int whole;        // one CTA per segment
};

template <int DIM>
constexpr int kSlot = 16 * DIM + 16;  // a part: outputs of 16 rows, their log2-sum-exp2

__device__ __forceinline__ int tiles_of(const Kv8Span& s) {
  return s.end > s.begin ? (s.end + kTile - 1) / kTile - s.begin / kTile : 0;
}

// a / b of numbers >= 0; nearly always both have 32 bits, whose division is far shorter
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
// Shares of the line of tiles: CTA c of n (at most 152), warp w of it.
struct Shares {
  int64_t each;
  uint32_t rest, n;
  __device__ __forceinline__ Shares(int64_t all, int64_t ctas) {
    each = quotient(all, ctas), n = (uint32_t)ctas, rest = (uint32_t)(all - each * ctas);
  }
  __device__ __forceinline__ int64_t start(int64_t c) const { return each * c + rest * (uint32_t)c / n; }
};
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
  c.h = n > 0 ? (int)quotient(off, n) : 0;
  c.u0 += c.h * n;
  c.tile = c.t0 + (int)(off - c.h * n);
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

// TWO: a page holds half a tile.  R8: at most eight query rows.
template <int MODE, int DIM, int S, bool TWO, bool R8>
__global__ void __launch_bounds__(kWarps * 32, 1)
    kv8_decode_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int KSTEPS = DIM / 16, NT = DIM / 8;      // 16-byte chunks of a row; n tiles of V
  constexpr int NE = R8 ? 1 : 2;                      // query rows of a thread: g, g + 8
  constexpr bool F8 = MODE == GDN_QDQ_E4M3;           // scores from the codes as they are
  constexpr float kRest = 32.f;                       // R8: of q's second part
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
      const Shares shares(all, n);
      const int64_t c0 = shares.start(blockIdx.x), c1 = shares.start(blockIdx.x + 1);
      lo = warp_start(c0, c1, warp), hi = warp_start(c0, c1, warp + 1);
      if (lo < hi) pc = locate(p, lo, lane);
    }
  }
  if (!a.whole && blockIdx.x == 0 && warp == 0) {
    // tiles before each row, for the join
    int64_t before = 0;
    for (int64_t r0 = 0; r0 < p.rows; r0 += 32) {
      int64_t mine = r0 + lane < p.rows ? tiles_of(kv8_span(p, r0 + lane)) : 0, x = mine;
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (r0 + lane < p.rows) a.before[r0 + lane] = before + x - mine;
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) a.before[p.rows] = before;
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
        const float2 sc = kv8_scales(p.scales[tile], p.scales[tile + p.pages * p.heads]);
        w_ks = sc.x, w_lv = sc.y;
      }
    }
    const int from = first - w_base;
    const int id0 = __shfl_sync(0xffffffffu, w_id, from);
    const float ks0 = __shfl_sync(0xffffffffu, w_ks, from), lv0 = __shfl_sync(0xffffffffu, w_lv, from);
    const int id1 = TWO ? __shfl_sync(0xffffffffu, w_id, from + 1) : id0;
    const float ks1 = TWO ? __shfl_sync(0xffffffffu, w_ks, from + 1) : ks0;
    const float lv1 = TWO ? __shfl_sync(0xffffffffu, w_lv, from + 1) : lv0;
    if (lane == 0) {
      meta[warp][st] = make_float4(ks0, lv0, ks1, lv1);
      valid[warp][st] = (id0 >= 0) | (id1 >= 0) << 1;
      unsigned char* k = ring + st * 2 * kBytes;
      constexpr int per = TWO ? kBytes / 2 : kBytes;
      mbar_expect_tx(&bars[warp][st],
                     (uint32_t)(per * 2 * ((id0 >= 0) + (TWO && id1 >= 0))));
      if (id0 >= 0) {
        const int z = id0 * p.heads + pc.h, y = j0 & (p.page - 1);
        tma_load_3d(k, &a.map, 0, y, z, &bars[warp][st]);
        tma_load_3d(k + kBytes, &a.map, 0, y, z + (int)(p.pages * p.heads), &bars[warp][st]);
      }
      if (TWO && id1 >= 0) {
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
  if (p.cu) kv8_fill<DIM>(p, (int64_t)blockIdx.x * kWarps + warp, (int64_t)gridDim.x * kWarps, lane);

  // ---- segments ----
  bool bad = false;
  int st = 0;
  uint32_t parity = 0;
  float oacc[NT][4];
  float lsum[NE], m[NE], mv[NE];
  Kv8Span sp;
  int64_t part = -1;  // segment left in registers at the end
  int64_t u_done = lo;
  for (int64_t u = lo; u < hi && !bad;) {
    const int64_t u0 = cc.u0, u1 = u0 + (cc.t1 - cc.t0);
    const int64_t stop = u1 < hi ? u1 : hi;
    sp = kv8_span(p, cc.r);
    const int rows = sp.n * p.group;
    // q fragments.  INT8: fp16, element pairs in the order kv8_half2 gives K's.  E4M3:
    // the two parts of q (kv8.cuh).  Up to eight rows (R8) the second ones are rows 8-15
    // of the same fragment, so E4M3 as well; with 2^5 of their own, which their sums give
    // back, that leaves 2^-15 where E5M2 leaves 2^-14.  Else they are E5M2 in a fragment of
    // their own.
    constexpr int QF = F8 ? (R8 ? DIM / 32 : DIM / 16) : KSTEPS;
    uint32_t qf[QF][4];
    float rowfac[NE];
    int beg[NE], end[NE];
    {
      uint2 raw[NE][KSTEPS];
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        float most = 0.f;
        const int i = g + 8 * e;
        const int qi = i / p.group;
        const bool have = i < rows;
        beg[e] = end[e] = 0;
        if (have) kv8_seen(p, sp, qi, beg[e], end[e]);
        const __nv_bfloat16* x = p.x + kv8_at(p, cc.r, sp.base, qi, p.x_row, p.x_token) +
                                 (cc.h * p.group + i % p.group) * p.x_head + 4 * t;
#pragma unroll
        for (int c = 0; c < KSTEPS; ++c) {
          raw[e][c] = have ? *reinterpret_cast<const uint2*>(x + 16 * c) : make_uint2(0, 0);
          float f[4];
          bf16x4(raw[e][c], f);
          most = fmaxf(most, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        float to, back;
        kv8_q_factor<F8 ? 7 : 8>(most, to, back);
        rowfac[e] = back * p.scale * kLog2eF;
#pragma unroll
        for (int c = 0; c < KSTEPS; ++c) {
          float f[4];
          bf16x4(raw[e][c], f);
          if constexpr (F8) {
            // k 16 c + 4 t ..: register 2 (c & 1) of row g, 2 (c & 1) + 1 of row g + 8
            float rest[4];
            const uint32_t hi = kv8_q_first(f, to, rest);
            if constexpr (R8) {
              float2 l0, l1;
              qf[c / 2][2 * (c & 1)] = hi;
              qf[c / 2][2 * (c & 1) + 1] = e4m3_code2(rest[0], rest[1], kRest, l0) |
                                           (uint32_t)e4m3_code2(rest[2], rest[3], kRest, l1) << 16;
            } else {
              qf[c / 2][2 * (c & 1) + e] = hi, qf[DIM / 32 + c / 2][2 * (c & 1) + e] = kv8_e5m2x4(rest);
            }
          } else {
            qf[c][e] = pack_f16(f[0] * to, f[2] * to);
            qf[c][2 + e] = pack_f16(f[1] * to, f[3] * to);
            if constexpr (R8) qf[c][1] = qf[c][3] = 0;
          }
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
#pragma unroll
    for (int e = 0; e < NE; ++e) lsum[e] = 0.f, m[e] = mv[e] = -INFINITY;

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
          if constexpr (F8) {
            mma_e4m3(s[j], qf[2 * q], r[0], r[1]);
            mma_e4m3(s[j], qf[2 * q + 1], r[2], r[3]);
            if constexpr (!R8) {
              mma_e5m2_e4m3(s[j], qf[DIM / 32 + 2 * q], r[0], r[1]);
              mma_e5m2_e4m3(s[j], qf[DIM / 32 + 2 * q + 1], r[2], r[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b0, b1;
              kv8_half2<MODE>(r[i], b0, b1);
              mma_f16(s[j], qf[4 * q + i], b0, b1);
            }
          }
        }
        if constexpr (F8 && R8)
          s[j][0] = fmaf(s[j][2], 1.f / kRest, s[j][0]), s[j][1] = fmaf(s[j][3], 1.f / kRest, s[j][1]);
      }
      const int j0 = cc.tile * kTile;
      const bool mask = have != 3 || j0 < in0 || j0 + kTile > in1;
      constexpr int H = TWO ? 2 : 1;  // blocks of the tile that have scales of their own
      float top[NE][H];
#pragma unroll
      for (int e = 0; e < NE; ++e) {
#pragma unroll
        for (int f = 0; f < H; ++f) {
          const float fac = rowfac[e] * (f ? sc.z : sc.x);
          float x = -INFINITY;
#pragma unroll
          for (int j = 4 / H * f; j < 4 / H * (f + 1); ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float y = s[j][2 * e + i] * fac;
              if (mask) {
                const int at = j0 + 8 * j + 2 * t + i;
                if (at < beg[e] || at >= end[e] || !(have >> f & 1)) y = -INFINITY;
              }
              s[j][2 * e + i] = y;
              x = fmaxf(x, y);
            }
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          top[e][f] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        }
      }
      float scale_o[NE];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        float nm = fmaxf(m[e], top[e][0]), nv = fmaxf(mv[e], top[e][0] + sc.y);
        if (TWO) nm = fmaxf(nm, top[e][H - 1]), nv = fmaxf(nv, top[e][H - 1] + sc.w);
        const float um = nm == -INFINITY ? 0.f : nm, uv = nv == -INFINITY ? 0.f : nv;
        lsum[e] *= ex2_approx_f(m[e] - um);
        scale_o[e] = ex2_approx_f(mv[e] - uv);
        moved |= nv != mv[e];
        float f_half[H];
        f_half[0] = ex2_approx_f(fminf(um + sc.y - uv, 126.f));
        if (TWO) f_half[H - 1] = ex2_approx_f(fminf(um + sc.w - uv, 126.f));
        m[e] = nm, mv[e] = nv;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w = ex2_approx_f(s[j][2 * e + i] - um);
            lsum[e] += w;
            s[j][2 * e + i] = w * f_half[TWO ? j / 2 : 0];
          }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          oacc[i][0] *= scale_o[0], oacc[i][1] *= scale_o[0];
          if constexpr (!R8) oacc[i][2] *= scale_o[NE - 1], oacc[i][3] *= scale_o[NE - 1];
        }
      }
      // ---- output: 16 keys per step; a 16-byte chunk of V gives two n tiles ----
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t pf[4];
        pf[0] = pack_f16(s[2 * k][0], s[2 * k][1]);
        pf[1] = R8 ? 0 : pack_f16(s[2 * k][2], s[2 * k][3]);
        pf[2] = pack_f16(s[2 * k + 1][0], s[2 * k + 1][1]);
        pf[3] = R8 ? 0 : pack_f16(s[2 * k + 1][2], s[2 * k + 1][3]);
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
    float lse2[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      float l = lsum[e];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      // l is 0 where no key is seen, and NaN where a score is
      lse2[e] = l == 0.f ? -INFINITY : m[e] + log2f(l);
      const float fac = kv8_out_factor<MODE>(mv[e], m[e], l);
#pragma unroll
      for (int i = 0; i < NT; ++i) oacc[i][2 * e] *= fac, oacc[i][2 * e + 1] *= fac;
    }
    const bool whole = lo <= u0 && u1 <= hi;
    if (whole || u1 < hi) {
#pragma unroll
      for (int e = 0; e < NE; ++e) {
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
#pragma unroll
      for (int e = 0; e < NE; ++e)
        if (t == 0) s_lse[warp][g + 8 * e] = lse2[e];
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
  grid_dep_launch();  // the join may be scheduled (it waits for the whole of this launch)
  if (lane == 0) s_u0[warp] = part;
  // every ring is done with; where a wait gave up the parts are not all there, and with a
  // CTA per segment, whose parts make a whole otherwise, there is no workspace for them
  if (__syncthreads_or(bad)) return;
  float* parts = reinterpret_cast<float*>(smem);  // [warp][16][DIM]
  if (part >= 0) {
#pragma unroll
    for (int e = 0; e < NE; ++e) {
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
        if (s_u0[w] == u0) top = max_nan(top, s_lse[w][i]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
      if (top != -INFINITY) {
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
      const float lse2 = top != -INFINITY ? top + log2f(l) : -INFINITY;
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

// Joins the parts of a segment that several CTAs hold, in order of the shares.  A
// CTA does some output rows of one segment (a part whose log-sum-exp is NaN makes the
// output NaN); with few parts a warp does a whole
// row, with many the warps take parts and their sums are added in warp order.
template <int DIM>
__global__ void __launch_bounds__(256) kv8_join_kernel(const __grid_constant__ DecodeArgs a, int grid) {
  constexpr int kList = 256, kFew = 12;
  __shared__ int s_at[kList];
  __shared__ float s_w[kList];
  __shared__ float red[8];
  __shared__ __align__(16) float s_o[8][DIM];
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int64_t r = blockIdx.x / p.heads;
  const int h = blockIdx.x % p.heads;
  const Kv8Span sp = kv8_span(p, r);
  const int n = tiles_of(sp), rows = sp.n * p.group;
  grid_dep_wait();  // by every CTA: the launches after this one are ordered behind it alone
  if (n == 0) return;
  const int64_t all = a.before[p.rows] * p.heads, ctas = ctas_for(all, grid);
  const int64_t u0 = a.before[r] * p.heads + (int64_t)h * n, u1 = u0 + n;
  // CTAs whose shares meet the segment: c with start(c) < u1 and start(c + 1) > u0
  const Shares shares(all, ctas);
  auto cta_of = [&](int64_t u) {
    const float near = (float)u * ((float)ctas / (float)all);
    int c = min((int)near, (int)ctas - 1);
    while (c > 0 && shares.start(c) > u) --c;
    while (shares.start(c + 1) <= u) ++c;
    return c;
  };
  const int64_t c0 = cta_of(u0), c1 = cta_of(u1 - 1);
  // one entry per CTA for what its warps left of the segment, and one for a warp
  // that goes on after the segment's end
  const int entries = (int)(c1 - c0 + 1) + 1;
  bool direct = false;
  if (tid < entries) {
    const bool after = tid == entries - 1;
    const int64_t c = after ? c1 : c0 + tid;
    const int64_t lo = shares.start(c), hi = shares.start(c + 1);
    int at = -1;
    int64_t first = -1, last_hi = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int64_t s = warp_start(lo, hi, w), e = warp_start(lo, hi, w + 1);
      if (s >= e || s >= u1 || e <= u0) continue;
      if (s <= u0 && e >= u1) {
        direct = true;
      } else if (e <= u1) {
        if (first < 0) {
          first = s;
          if (!after) at = (int)((c * kWarps + w) * 2 + 1);
        }
        last_hi = e;
      } else if (after) {
        at = (int)((c * kWarps + w) * 2);
      }
    }
    if (first >= 0 && first <= u0 && last_hi >= u1) direct = true;
    s_at[tid] = at;
  }
  if (__syncthreads_or(direct)) return;  // written already
  auto lse_of = [&](int k, int i) {
    return s_at[k] >= 0 ? a.ws[(int64_t)s_at[k] * kSlot<DIM> + 16 * DIM + i] : -INFINITY;
  };
  auto add = [&](int k, int i, float c, float4& o) {
    if (lane < DIM / 4) {
      const float4 x = *reinterpret_cast<const float4*>(a.ws + (int64_t)s_at[k] * kSlot<DIM> + i * DIM + 4 * lane);
      o.x = fmaf(c, x.x, o.x), o.y = fmaf(c, x.y, o.y), o.z = fmaf(c, x.z, o.z), o.w = fmaf(c, x.w, o.w);
    }
  };
  auto finish = [&](int i, float4 o, float top, float l) {
    const int64_t to = out_row<DIM>(p, sp, h, i);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane < DIM / 4)
      *reinterpret_cast<uint2*>(p.o + to * DIM + 4 * lane) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (p.lse && lane == 0) p.lse[to] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
  };
  if (entries <= kFew) {
    for (int i = blockIdx.y * 8 + warp; i < rows; i += gridDim.y * 8) {
      const float mine = lane < entries ? lse_of(lane, i) : -INFINITY;
      float top = mine;
      for (int d = 16; d; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float l = 0.f;
      if (top != -INFINITY)
        for (int k = 0; k < entries; ++k) {
          if (s_at[k] < 0) continue;
          const float c = ex2_approx_f(__shfl_sync(0xffffffffu, mine, k) - top);
          l += c;
          add(k, i, c, o);
        }
      finish(i, o, top, l);
    }
    return;
  }
  for (int i = blockIdx.y; i < rows; i += gridDim.y) {
    float top = tid < entries ? lse_of(tid, i) : -INFINITY;
    const float mine = top;
    for (int d = 16; d; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    __syncthreads();
    if (lane == 0) red[warp] = top;
    __syncthreads();
    for (int w = 0; w < 8; ++w) top = max_nan(top, red[w]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    __syncthreads();
    if (tid < entries) s_w[tid] = s_at[tid] >= 0 && top != -INFINITY ? ex2_approx_f(mine - top) : 0.f;
    __syncthreads();
    // four parts at a time, so that their loads are in flight together
    for (int k0 = warp; k0 < entries; k0 += 32) {
      float c[4];
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = k0 + 8 * j;
        c[j] = e < entries ? s_w[e] : 0.f;
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c[j] > 0.f && lane < DIM / 4)
          x[j] = *reinterpret_cast<const float4*>(a.ws + (int64_t)s_at[e] * kSlot<DIM> + i * DIM + 4 * lane);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l += c[j];
        o.x = fmaf(c[j], x[j].x, o.x), o.y = fmaf(c[j], x[j].y, o.y);
        o.z = fmaf(c[j], x[j].z, o.z), o.w = fmaf(c[j], x[j].w, o.w);
      }
    }
    __syncthreads();
    if (lane < DIM / 4) *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = o;
    if (lane == 0) red[warp] = l;
    __syncthreads();
    if (warp == 0) {
      l = 0.f, o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < 8; ++w) {
        l += red[w];
        if (lane < DIM / 4) {
          const float4 x = *reinterpret_cast<const float4*>(&s_o[w][4 * lane]);
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
        }
      }
      finish(i, o, top, l);
    }
  }
}

// Most tiles that a row can have, by its table and window.
int64_t most_tiles(const Kv8Params& p) {
  int64_t keys = (int64_t)p.cols * p.page;
  if (p.window > 0 && (int64_t)p.window + p.tokens < keys) keys = (int64_t)p.window + p.tokens;
  return (keys + kTile - 1) / kTile + 1;
}
// One CTA per segment, or the line of all tiles?  A CTA alone takes 6 us + 0.18 us per
// tile; the line pays for its shares and a second launch, but
// leaves no SM idle and no wave half full.  Measured, line / segment in us, 128-wide
// E4M3 heads (INT8 within 8 % of these):
//     segments     256 keys   1024 keys   2048 keys   4096 keys
//           2     10.1/7.2   11.9/11.5   13.4/17.5   11.9/29.3
//           8     10.1/7.0   12.3/11.4   13.4/17.2   12.1/29.1
//          64     10.9/7.5   18.2/11.7   20.7/17.8   25.4/29.5
//         152     12.3/7.4   17.2/12.3   23.4/18.6   38.3/33.7
//         256     17.7/13.4  25.2/22.8   39.7/39.6   59.0/63.4
//         512     21.8/25.0  40.4/49.7   59.5/76.3   98.9/122
//        8192      151/357     390/617
// and 64-wide E4M3 heads (INT8 within 8 %):
//           2      9.1/6.4   11.3/9.5   12.1/13.5  10.9/21.6
//          64     10.3/6.6   15.9/9.7   17.5/13.8  20.3/22.2
//         152     10.9/6.6   14.3/9.7   18.3/13.8  26.8/22.5
//         256     16.0/11.7  20.9/17.9  27.5/26.3  45.2/47.1
//         512     18.9/21.8  29.1/34.1  46.0/57.9  73.7/90.9
// So: one wave up to a length that grows with the SMs it fills, two waves of
// short segments, and the line for the rest (of the above it misses 5 % once: 64-wide,
// 256 segments of 2048 keys).
bool by_segment(const Kv8Params& p) {
  const int64_t segments = p.rows * p.heads, tiles = most_tiles(p);
  return segments <= 152 ? tiles <= 36 + segments : segments <= 304 && tiles <= 40;
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
  // up to eight query rows: half of the softmax's work, and q's two parts in one
  // fragment (eight rows, 64 rows of 2192 .. 8192 keys, 8 heads, both launches: E4M3 121 us,
  // with the code for sixteen 162; INT8 129 and 139)
  const bool r8 = (int64_t)p.tokens * p.group <= 8;
  auto kern = p.page < kTile
                  ? (r8 ? kv8_decode_kernel<MODE, DIM, S, true, true> : kv8_decode_kernel<MODE, DIM, S, true, false>)
                  : (r8 ? kv8_decode_kernel<MODE, DIM, S, false, true> : kv8_decode_kernel<MODE, DIM, S, false, false>);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return GDN_ERR_CUDA;
  kern<<<(unsigned)grid, kWarps * 32, bytes, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  if (a.whole) return GDN_OK;
  // rows of a segment in one CTA, unless the segments leave SMs idle
  const int64_t segments = p.rows * p.heads, rows = (int64_t)p.tokens * p.group;
  int64_t y = 304 / segments;
  y = y < rows ? y : rows;
  y = y < 1 ? 1 : y;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)segments, (unsigned)y);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_join_kernel<DIM>, a, (int)grid) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Workspace: tiles before each row, then the parts.
size_t before_bytes(const Kv8Params& p) { return ((size_t)(p.rows + 1) * 8 + 255) / 256 * 256; }

}  // namespace

size_t kv8_decode_workspace(const Kv8Params& p, int dim) {
  if (by_segment(p)) return 0;
  return before_bytes(p) + (size_t)grid_of(p) * kWarps * 2 * (16 * dim + 16) * sizeof(float);
}

gdn_status launch_kv8_decode(const Kv8Params& p, int mode, int dim, void* workspace,
                             cudaStream_t st) {
  DecodeArgs a;
  a.p = p;
  a.before = static_cast<int64_t*>(workspace);
  a.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + before_bytes(p));
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
