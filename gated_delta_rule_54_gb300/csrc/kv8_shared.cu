// Attention over the 8-bit paged cache where the rows of a group have their first tokens in
// common.
//
// A CTA takes 16 query rows of a (row, K/V head): its warps go through tiles of 32 keys, the
// group's (pages of the group's first row) and then the row's own, each from registers, and
// their parts are joined in shared memory.
//
// Codes go from global memory into the lanes that need them.  A score is a sum over dims in
// any order, so a lane's 16 bytes of a key are four steps of a warp product whose other operand,
// q, is laid out alike; and the columns of P V are dims in any order, so a lane's 16 bytes
// of each of four keys are its column of 16 products, after an exchange of bytes between
// neighbouring keys.
#include <cuda.h>

#include "kv8.cuh"
#include "launch.h"

namespace gdn {

namespace {

constexpr int kTile = 32, kWarps = 4;

struct SharedArgs {
  Kv8Params p;
  const int32_t* shared;
  int beams;
};

// Keys of query i of a row (all of them, of the whole row): [0, end).
__device__ __forceinline__ int seen_end(const Kv8Params& p, int64_t len, int i) {
  const int64_t pos = len - p.tokens + i;
  const int64_t most = (int64_t)p.cols * p.page;
  const int all = kv8_clamp(len, 0, most);
  return p.causal ? kv8_clamp(pos + 1, 0, all) : pos < 0 ? 0 : all;
}

// 16 bytes (or 8) of codes
template <int DIM>
struct Codes {
  using T = uint4;
};
template <>
struct Codes<64> {
  using T = uint2;
};

// ROWS: 16 or 8 query rows of the CTA.
template <int MODE, int DIM, int ROWS>
__global__ void __launch_bounds__(kWarps * 32) kv8_own_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int NE = ROWS / 8, KC = DIM / 64, KSTEPS = DIM / 16, NT = DIM / 8;
  using V = typename Codes<DIM>::T;
  __shared__ __align__(16) float s_o[kWarps][ROWS][DIM];
  __shared__ float s_lse[kWarps][ROWS];
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  const int64_t r = blockIdx.x / p.heads;
  const int h = blockIdx.x % p.heads, i0 = blockIdx.y * ROWS, rows = min(p.tokens * p.group - i0, ROWS);
  const int64_t len = p.lengths[r];
  const int most = kv8_clamp(len, 0, (int64_t)p.cols * p.page);
  const int common = kv8_clamp(a.shared[r / a.beams], 0, most);
  const int32_t *own = p.table + r * p.cols, *group = p.table + r / a.beams * a.beams * p.cols;

  // ---- queries: fp16 by a power of two per row, in the order of the codes ----
  uint32_t qf[KSTEPS][4];
  float rowfac[NE];
  int end[NE];
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    const int i = i0 + g + 8 * e;
    const bool have = g + 8 * e < rows;
    end[e] = have ? seen_end(p, len, i / p.group) : 0;
    const __nv_bfloat16* x = p.x + r * p.x_row + (i / p.group) * p.x_token + (int64_t)(h * p.group + i % p.group) * p.x_head;
    uint2 raw[KSTEPS];
    float mx = 0.f;
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      // step s: the four dims from 64 (s / 4) + 16 t + 4 (s % 4) on
      raw[s] = have ? *reinterpret_cast<const uint2*>(x + 64 * (s / 4) + 16 * t + 4 * (s % 4)) : make_uint2(0, 0);
      float f[4];
      bf16x4(raw[s], f);
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    float to, back;
    kv8_q_factor<8>(mx, to, back);
    rowfac[e] = back * p.scale * kLog2eF * (MODE == GDN_QDQ_E4M3 ? 256.f : 1.f);
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      float f[4];
      bf16x4(raw[s], f);
      qf[s][e] = pack_f16(f[0] * to, f[2] * to);
      qf[s][2 + e] = pack_f16(f[1] * to, f[3] * to);
    }
  }
  if constexpr (NE == 1) {
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) qf[s][1] = qf[s][3] = 0;
  }

  float oacc[NT][4], lsum[NE], m[NE], mv[NE];
#pragma unroll
  for (int i = 0; i < NT; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;
#pragma unroll
  for (int e = 0; e < NE; ++e) lsum[e] = 0.f, m[e] = mv[e] = -INFINITY;

  // ---- keys: first the group's, then the row's own ----
  for (int part = 0; part < 2; ++part) {
    const int from = part ? common : 0, to = part ? most : common;
    const int32_t* pages = part ? own : group;
    const int t0 = from / kTile, t1 = to > from ? (to + kTile - 1) / kTile : t0;
    for (int tile = t0 + warp; tile < t1; tile += kWarps) {
      const int j0 = tile * kTile;
      int64_t block[2];
      bool have[2];
      float ks[2], lv[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int j = j0 + 16 * f;
        const int id = j < to && (j >> p.shift) < p.cols ? pages[j >> p.shift] : -1;
        have[f] = id >= 0 && id < p.pages;
        block[f] = (int64_t)(have[f] ? id : 0) * p.heads + h;
        ks[f] = 0.f, lv[f] = -INFINITY;
        if (have[f]) {
          const float2 sc = kv8_scales(p.scales[block[f]], p.scales[block[f] + p.pages * p.heads]);
          ks[f] = sc.x, lv[f] = sc.y;
        }
      }
      uint4 kc[4][KC];
      V vc[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          kc[j][c] = make_uint4(0, 0, 0, 0);
          if (have[j / 2])
            kc[j][c] = __ldg(reinterpret_cast<const uint4*>(
                p.codes + (block[j / 2] * p.page + ((j0 + 8 * j + g) & (p.page - 1))) * DIM + 64 * c + 16 * t));
        }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          vc[k][x] = V();
          if (have[k])
            vc[k][x] = __ldg(reinterpret_cast<const V*>(
                p.codes + ((block[k] + p.pages * p.heads) * p.page +
                           ((j0 + 16 * k + 2 * t + (x & 1) + 8 * (x >> 1)) & (p.page - 1))) * DIM + DIM / 8 * g));
        }
      // ---- scores: n tile j = keys 8 j .. 8 j + 7 ----
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint32_t w[4] = {kc[j][c].x, kc[j][c].y, kc[j][c].z, kc[j][c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b0, b1;
            kv8_half2<MODE>(w[i], b0, b1);
            mma_f16(s[j], qf[4 * c + i], b0, b1);
          }
        }
      }
      float top[NE][2];
#pragma unroll
      for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float fac = rowfac[e] * ks[f];
          float x = -INFINITY;
#pragma unroll
          for (int j = 2 * f; j < 2 * f + 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int at = j0 + 8 * j + 2 * t + i;
              float y = s[j][2 * e + i] * fac;
              if (at < from || at >= to || at >= end[e] || !have[f]) y = -INFINITY;
              s[j][2 * e + i] = y;
              x = fmaxf(x, y);
            }
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          top[e][f] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        }
      // ---- softmax: m the largest score, mv the largest score + log2 of V's scale ----
      float by[NE];
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const float nm = fmaxf(m[e], fmaxf(top[e][0], top[e][1]));
        const float nv = fmaxf(mv[e], fmaxf(top[e][0] + lv[0], top[e][1] + lv[1]));
        const float um = nm == -INFINITY ? 0.f : nm, uv = nv == -INFINITY ? 0.f : nv;
        lsum[e] *= ex2_approx_f(m[e] - um);
        by[e] = ex2_approx_f(mv[e] - uv);
        m[e] = nm, mv[e] = nv;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float half = ex2_approx_f(fminf(um + lv[f] - uv, 126.f));
#pragma unroll
          for (int j = 2 * f; j < 2 * f + 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float w = ex2_approx_f(s[j][2 * e + i] - um);
              lsum[e] += w;
              s[j][2 * e + i] = w * half;
            }
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        oacc[i][0] *= by[0], oacc[i][1] *= by[0];
        if constexpr (NE == 2) oacc[i][2] *= by[1], oacc[i][3] *= by[1];
      }
      // ---- output: n tile j = dims j, j + DIM / 8, ... ----
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t pf[4];
        pf[0] = pack_f16(s[2 * k][0], s[2 * k][1]);
        pf[1] = NE == 2 ? pack_f16(s[2 * k][2], s[2 * k][3]) : 0;
        pf[2] = pack_f16(s[2 * k + 1][0], s[2 * k + 1][1]);
        pf[3] = NE == 2 ? pack_f16(s[2 * k + 1][2], s[2 * k + 1][3]) : 0;
        const uint32_t* w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = reinterpret_cast<const uint32_t*>(&vc[k][x]);
#pragma unroll
        for (int i = 0; i < DIM / 32; ++i)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            // bytes of two neighbouring keys: (a0 a1 b0 b1), then (a2 a3 b2 b3)
            uint32_t e0, o0, e1, o1;
            kv8_half2<MODE>(__byte_perm(w[0][i], w[1][i], z ? 0x7632 : 0x5410), e0, o0);
            kv8_half2<MODE>(__byte_perm(w[2][i], w[3][i], z ? 0x7632 : 0x5410), e1, o1);
            mma_f16(oacc[4 * i + 2 * z], pf, e0, e1);
            mma_f16(oacc[4 * i + 2 * z + 1], pf, o0, o1);
          }
      }
    }
  }

  // ---- the warps' parts: outputs over their own keys, and log2 of the sums ----
#pragma unroll
  for (int e = 0; e < NE; ++e) {
    float l = lsum[e];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float fac = kv8_out_factor<MODE>(mv[e], m[e], l);
    if (t == 0) s_lse[warp][g + 8 * e] = l == 0.f ? -INFINITY : m[e] + log2f(l);
    // columns 2 t and 2 t + 1 of n tile j: dims DIM / 8 (2 t) + j and DIM / 8 (2 t + 1) + j
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < NT; j += 4)
        *reinterpret_cast<float4*>(&s_o[warp][g + 8 * e][DIM / 8 * (2 * t + c) + j]) =
            make_float4(oacc[j][2 * e + c] * fac, oacc[j + 1][2 * e + c] * fac, oacc[j + 2][2 * e + c] * fac,
                        oacc[j + 3][2 * e + c] * fac);
  }
  __syncthreads();
  for (int i = warp; i < rows; i += kWarps) {
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = max_nan(top, s_lse[w][i]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int w = 0; w < kWarps && top != -INFINITY; ++w) {
      const float c = ex2_approx_f(s_lse[w][i] - top);
      l += c;
      if (lane < DIM / 4) {
        const float4 x = *reinterpret_cast<const float4*>(&s_o[w][i][4 * lane]);
        o.x = fmaf(c, x.x, o.x), o.y = fmaf(c, x.y, o.y), o.z = fmaf(c, x.z, o.z), o.w = fmaf(c, x.w, o.w);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = (r * p.tokens + (i0 + i) / p.group) * (p.heads * p.group) + h * p.group + (i0 + i) % p.group;
    if (lane < DIM / 4)
      *reinterpret_cast<uint2*>(p.o + at * DIM + 4 * lane) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
  }
}

template <int MODE, int DIM>
gdn_status run(const SharedArgs& a, cudaStream_t st) {
  const Kv8Params& p = a.p;
  const int64_t rows = (int64_t)p.tokens * p.group;
  const bool few = rows <= 8;
  const int64_t y = few ? 1 : (rows + 15) / 16;
  if (y > 65535) return GDN_ERR_UNSUPPORTED_SHAPE;
  const dim3 grid((unsigned)(p.rows * p.heads), (unsigned)y);
  if (few) kv8_own_kernel<MODE, DIM, 8><<<grid, kWarps * 32, 0, st>>>(a);
  else kv8_own_kernel<MODE, DIM, 16><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

size_t kv8_shared_workspace(const Kv8Params&, int, int) { return 0; }

gdn_status launch_kv8_shared(const Kv8Params& p, int beams, const int32_t* shared, int mode, int dim,
                             void*, cudaStream_t st) {
  SharedArgs a;
  a.p = p;
  a.shared = shared, a.beams = beams;
  if (mode == GDN_QDQ_E4M3) return dim == 128 ? run<GDN_QDQ_E4M3, 128>(a, st) : run<GDN_QDQ_E4M3, 64>(a, st);
  return dim == 128 ? run<GDN_QDQ_INT8, 128>(a, st) : run<GDN_QDQ_INT8, 64>(a, st);
}

}  // namespace gdn
