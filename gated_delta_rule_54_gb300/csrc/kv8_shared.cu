// Attention over the 8-bit paged cache where the rows of a group have their first tokens in
// common.  Two launches: the group's tokens, once for all its rows, on the tensor cores; then
// each row's own tokens, and the join of both.
//
// The group's tokens.  The query rows of a (group, K/V head) are its rows times their
// queries times the query heads that share the head; they are few, so the products are laid
// out with the keys as the long side.  Per 128 keys and up to NQ query rows:
//     S = K Q^T      (tcgen05, fp16 -> fp32 in TMEM: lane = key, column = query)
//     P = 2^(s - reference), fp16 to shared memory
//     O += V^T P     (lane = dim, column = query)
// and only the columns in use cost exponentials.  All tiles of all (group, head, block of query
// rows) form one line, of which every CTA takes an equal, contiguous share; what it has of a
// (group, head, block) is a part: outputs over its own keys, and their log-sum-exp.
// One warp brings the codes of a tile by TMA (a box per page), four turn K's into fp16 (exact)
// and four V's, one lane issues the products, and eight warps are the keys: a thread
// has one key, and half of the queries.
//
// A column's maxima (of s, and of s + log2 of V's scale, which is one for 16 lanes) come by exchanges
// within half-warps and through shared memory.  The references follow them, per column, only
// when they grow by more than 2^8, which fp16 has the room for; so a row's result does not
// depend on the rows beside it.
//
// A row's own tokens.  A CTA takes 16 query rows of a (row, K/V head): its warps go through
// tiles of 32 keys from registers, and their parts are joined with those of the group's tokens.
// Codes go from global memory into the lanes that need them.  A score is a sum over dims in
// any order, so a lane's 16 bytes of a key are four steps of a warp product whose other operand,
// q, is laid out alike; and the columns of P V are dims in any order, so a lane's 16 bytes
// of each of four keys are its column of 16 products, after an exchange of bytes between
// neighbouring keys.
#include <cuda.h>

#include "kv8_tc.cuh"
#include "launch.h"

namespace gdn {

namespace {

__device__ int g_kv8_shared_error;

constexpr int kTile = 32, kWarps = 4;  // own tokens: keys of a tile, warps of a CTA
constexpr int kKeys = 128;             // the group's tokens: keys of a tile
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kIssuer = kSoftWarps + 2 * kConvWarps, kLoader = kIssuer + 1;
constexpr int kThreads = 640;
// registers per thread of the warpgroups: together no more than the launch gave (5 x 96)
constexpr int kSoftRegs = 152, kConvRegs = 56, kRestRegs = 56;
static_assert(2 * kSoftRegs + 2 * kConvRegs + kRestRegs <= 5 * 96, "register shares");

struct SharedArgs {
  Kv8Params p;
  CUtensorMap map;  // codes, a page of a head per box
  const int32_t* shared;
  float *parts, *lses;  // [slot][stride][DIM], [slot][stride]
  int beams, nq, blocks;  // query rows of a block; blocks of a (group, head)
  int stride;             // query rows of a part
  int grid;               // CTAs of the first launch
};

// What kv8_half2 leaves out of K goes half to the query's factor and half to K's scale, so that
// neither leaves its range before the other.
template <int MODE>
constexpr float kRoot = MODE == GDN_QDQ_E4M3 ? 16.f : 1.f;

// Keys of query i of a row (all of them, of the whole row): [0, end).
__device__ __forceinline__ int seen_end(const Kv8Params& p, int64_t len, int i) {
  const int64_t pos = len - p.tokens + i;
  const int64_t most = (int64_t)p.cols * p.page;
  const int all = kv8_clamp(len, 0, most);
  return p.causal ? kv8_clamp(pos + 1, 0, all) : pos < 0 ? 0 : all;
}

// Tokens that a group has in common, and their tiles.
__device__ __forceinline__ int common_of(const SharedArgs& a, int64_t g) {
  return kv8_clamp(a.shared[g], 0, (int64_t)a.p.cols * a.p.page);
}
__device__ __forceinline__ int tiles_of(int keys) { return (int)(((int64_t)keys + kKeys - 1) / kKeys); }

// Tiles of groups [0, g1), counted for one (head, block).
__device__ __forceinline__ int64_t tiles_before(const SharedArgs& a, int64_t g1, int lane) {
  int64_t n = 0;
  for (int64_t g = lane; g < g1; g += 32) n += tiles_of(common_of(a, g));
  for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
  return n;
}

// Equal shares of the line of `all` tiles: the first `rest` of n CTAs have one tile more.
struct Shares {
  int64_t each, rest, n;
  __device__ __forceinline__ Shares(int64_t all, int grid) {
    n = all < grid ? all : grid;
    each = n > 0 ? all / n : 0, rest = n > 0 ? all - each * n : 0;
  }
  __device__ __forceinline__ int64_t start(int64_t c) const { return each * c + (c < rest ? c : rest); }
  __device__ __forceinline__ int64_t cta_of(int64_t u) const {
    const int64_t longer = rest * (each + 1);
    return u < longer ? u / (each + 1) : rest + (u - longer) / each;
  }
};

// A CTA's way through its share: pieces of (group, head, block).
struct Walk {
  int64_t left, g;
  int common, tiles, hq, t;  // of the group; head * blocks + block; tile
  __device__ __forceinline__ Walk(const SharedArgs& a, int64_t cta, int lane) {
    const int64_t groups = a.p.rows / a.beams, per = (int64_t)a.p.heads * a.blocks;
    const Shares s(tiles_before(a, groups, lane) * per, a.grid);
    left = 0, g = 0, common = tiles = hq = t = 0;
    if (cta >= s.n) return;
    const int64_t u = s.start(cta);
    left = s.start(cta + 1) - u;
    int64_t before = 0;
    for (int64_t g0 = 0;; g0 += 32) {
      const int64_t mine = g0 + lane < groups ? tiles_of(common_of(a, g0 + lane)) * per : 0;
      int64_t x = mine;
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + x > u);
      if (hit) {
        const int at = __ffs(hit) - 1;
        g = g0 + at;
        before += __shfl_sync(0xffffffffu, x - mine, at);
        break;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    common = common_of(a, g), tiles = tiles_of(common);
    const int64_t in = u - before;
    hq = (int)(in / tiles), t = (int)(in - (int64_t)hq * tiles);
  }
  // tiles of the piece
  __device__ __forceinline__ int count() const { return left < tiles - t ? (int)left : tiles - t; }
  __device__ __forceinline__ void next(const SharedArgs& a) {
    const int n = count();
    left -= n, t += n;
    if (t < tiles || left == 0) return;
    t = 0;
    if (++hq < a.p.heads * a.blocks) return;
    hq = 0;
    do common = common_of(a, ++g), tiles = tiles_of(common);
    while (tiles == 0);
  }
  __device__ __forceinline__ int64_t slot(const SharedArgs& a, int64_t cta) const {
    return g * a.p.heads * a.blocks + hq + cta;
  }
};

// Unit u (16 bytes = 8 columns) of a row of a tile in panels of 64 columns, `rows` rows each.
// Columns are stored in the order in which kv8_half2 gives them: of each four, 0 2 1 3.
__device__ __forceinline__ uint32_t unit_at(int row, int u, int rows) {
  return (uint32_t)((u >> 3) * (rows * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4));
}

// Of each of 16 columns the maximum (or sum) over the 16 lanes of a half-warp: lane l gets
// column l % 16.
template <bool SUM>
__device__ __forceinline__ float half_reduce(float (&x)[16], int lane) {
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      x[i] = SUM ? keep + got : fmaxf(keep, got);
    }
  }
  return x[0];
}

__device__ __forceinline__ void half_sync(int half) {
  asm volatile("bar.sync %0, 128;\n" ::"r"(1 + half) : "memory");
}
// the same, and whether any of the threads says yes
__device__ __forceinline__ bool half_any(int half, bool yes) {
  uint32_t any;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(any)
               : "r"((uint32_t)yes), "r"(1 + half)
               : "memory");
  return any;
}

// Shared memory of the first kernel: fp16 tiles K 0, K 1, V 0, V 1; the codes of the next ones
// arrive on their second panels, or, with 64 dims, behind.  V with 64 dims has a panel of zeros for
// the other 64 lanes of O.
template <int DIM, int NQ>
struct Room {
  static constexpr int tile = kKeys * DIM * 2, k = 0, v = 2 * tile, zero = 4 * tile;
  static constexpr int codes = zero + (DIM == 64 ? kKeys * 128 : 0);
  static constexpr int q = codes + (DIM == 64 ? 4 * kKeys * DIM : 0), pt = q + NQ * DIM * 2;
  static constexpr int bytes = pt + NQ / 64 * kKeys * 128 + 1024;
  static constexpr int codes_at(int kv, int b) {
    return DIM == 128 ? (2 * kv + b) * tile + kKeys * 128 : codes + (2 * kv + b) * kKeys * DIM;
  }
};

template <int MODE, int DIM, int NQ>
__global__ void __launch_bounds__(kThreads, 1) kv8_common_kernel(const __grid_constant__ SharedArgs a) {
  using R = Room<DIM, NQ>;
  constexpr uint32_t kCols = NQ == 64 ? 256 : 512;  // S 0, S 1, O
  constexpr uint32_t kIdQK = idesc_f16(128, NQ, 0, 0), kIdPV = idesc_f16(128, NQ, 1, 1);
  constexpr int kChunks = NQ / 32;  // of 16 columns, of a thread
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t cfull[2][2];                       // codes of K, of V; by buffer
  __shared__ __align__(8) uint64_t kfull[2], kfree[2], vfull[2], vfree[2];
  __shared__ __align__(8) uint64_t sfull[2], sfree[2], qready, pready, odone;
  __shared__ float2 meta[4][8];  // per 16 keys of a tile: K scale, log2 of V scale
  __shared__ int valid[4];       // bit c: they have a page
  __shared__ int s_lim[NQ], s_min[2];  // keys that a column sees; the fewest of a half's columns
  __shared__ __align__(16) float s_fac[NQ], s_m[NQ], s_out[NQ], s_by[2][NQ];
  __shared__ float s_mv[NQ];
  __shared__ __align__(16) float s_ratio[kSoftWarps][2][NQ / 2];  // 2^(log2 vs + m - mv), per half-warp
  __shared__ float2 s_red[4][NQ];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);  // uniform
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);

  grid_dep_launch();  // the rows' own tokens need nothing of this launch until their join
  if (warp == 0) tmem_alloc(&tmem_slot, kCols);
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cfull[0][i], 1), mbar_init(&cfull[1][i], 1);
      mbar_init(&kfull[i], kConvWarps * 32), mbar_init(&vfull[i], kConvWarps * 32);
      mbar_init(&kfree[i], 1), mbar_init(&vfree[i], 1);
      mbar_init(&sfull[i], 1), mbar_init(&sfree[i], kSoftWarps * 32);
    }
    mbar_init(&qready, kSoftWarps * 32), mbar_init(&pready, kSoftWarps * 32), mbar_init(&odone, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (DIM == 64) {
    for (int i = tid; i < kKeys * 8; i += kThreads) reinterpret_cast<uint4*>(smem + R::zero)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
  }
  Walk w(a, blockIdx.x, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // every wait is bounded, so when one gives up the other roles' do as well
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_wait(bar, parity)) return true;
    abort_flag = 1;
    return false;
  };
  auto all_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

  if (warp < kSoftWarps) {
    set_regs_up<kSoftRegs>();
    // ======================= keys =======================
    const int half = warp / 4, quad = warp & 3, key = quad * 32 + lane, sub = lane >> 4;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    unsigned char *sQ = smem + R::q, *sP = smem + R::pt;
    const int per_row = p.tokens * p.group, all_q = a.beams * per_row;
    bool ok = true;
    uint32_t n = 0;  // tiles so far
    for (; w.left > 0; w.next(a)) {
      const int nt = w.count(), h = w.hq / a.blocks, q0 = w.hq % a.blocks * NQ;
      const int here = min(all_q - q0, NQ);          // columns in use
      const int hc = (here + 31) / 32 * 16, c0 = half * hc;  // a half's, in chunks of 16; the first of mine
      // ---- queries: DIM / 8 lanes to a row ----
      {
        constexpr int kLanes = DIM / 8, kAt = 32 / kLanes;
        for (int c = warp * kAt + lane / kLanes; c < 2 * hc; c += kSoftWarps * kAt) {
          const int i = q0 + c, r_in = i / per_row, x_in = i - r_in * per_row, u = lane % kLanes;
          const int64_t r = w.g * a.beams + r_in;
          uint4 raw = make_uint4(0, 0, 0, 0);
          if (c < here)
            raw = __ldg(reinterpret_cast<const uint4*>(p.x + r * p.x_row + (x_in / p.group) * p.x_token +
                                                       (int64_t)(h * p.group + x_in % p.group) * p.x_head + 8 * u));
          float f[8], most = 0.f;
          bf16x8(raw, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[e]));
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
          float up, back;
          kv8_q_factor<8>(most, up, back);
          if (u == 0) {
            s_fac[c] = back * fabsf(p.scale) * kLog2eF * kRoot<MODE>;
            s_lim[c] = c < here ? min(seen_end(p, p.lengths[r], x_in / p.group), w.common) : 0;
          }
          if (p.scale < 0.f) up = -up;
          *reinterpret_cast<uint4*>(sQ + unit_at(c, u, NQ)) =
              make_uint4(pack_f16(f[0] * up, f[2] * up), pack_f16(f[1] * up, f[3] * up),
                         pack_f16(f[4] * up, f[6] * up), pack_f16(f[5] * up, f[7] * up));
        }
        fence_proxy_async();
        if (ok) mbar_arrive(&qready);
      }
      asm volatile("bar.sync 3, 256;\n" ::: "memory");  // both halves: the columns' limits and factors
      if (quad == 0) {
        int least = 0x7fffffff;
        for (int c = lane; c < hc; c += 32)
          if (c0 + c < here) least = min(least, s_lim[c0 + c]);
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) s_min[half] = least;
        for (int c = lane; c < hc; c += 32) s_m[c0 + c] = s_mv[c0 + c] = -INFINITY;
      }
      half_sync(half);
      const int least = s_min[half];
      float sum[kChunks][16];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[c][e] = 0.f;

      for (int i = 0; i < nt; ++i, ++n) {
        ok = ok && all_wait(&sfull[n & 1], (n >> 1) & 1);
        if (!ok) {  // a wait gave up: only the barriers that others may stand at
          half_sync(half);
          half_any(half, false);
          continue;
        }
        tc_fence_after();
        const uint32_t s_col = lanes + (n & 1) * NQ + c0;
        const int j0 = (w.t + i) * kKeys, at = j0 + key;
        const float2 sc = meta[n & 3][key >> 4];
        const bool there = valid[n & 3] >> (key >> 4) & 1;
        const bool mask = valid[n & 3] != 255 || j0 + kKeys > least;
        // ---- maxima ----
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (16 * c >= hc) break;
          float v[16];
          tmem_ld16(s_col + 16 * c, v);
          if (mask) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!there || at >= s_lim[c0 + 16 * c + e]) v[e] = -INFINITY;
          }
          const float x = half_reduce<false>(v, lane);
          const int col = c0 + 16 * c + (lane & 15);
          // (a factor of 0 would make -inf a NaN)
          float nm = x == -INFINITY ? x : x * (sc.x * s_fac[col]);
          float nv = nm + sc.y;
          nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 16));
          nv = fmaxf(nv, __shfl_xor_sync(0xffffffffu, nv, 16));
          if (lane < 16) s_red[quad][col] = make_float2(nm, nv);
        }
        half_sync(half);
        bool moved = false;
        for (int c = quad * 32 + lane; c < hc; c += 128) {
          const int col = c0 + c;
          float nm = -INFINITY, nv = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) nm = fmaxf(nm, s_red[q][col].x), nv = fmaxf(nv, s_red[q][col].y);
          const float m = s_m[col], mv = s_mv[col];
          float by = 1.f, by_o = 1.f;
          if (nm > m + 8.f) by = ex2_approx_f(m - nm), s_m[col] = nm, moved = true;
          if (nv > mv + 8.f) by_o = ex2_approx_f(mv - nv), s_mv[col] = nv, moved = true;
          s_by[0][col] = by, s_by[1][col] = by_o;
        }
        moved = half_any(half, moved);
        // ---- what the references' change makes of the sums so far ----
        if (n > 0 && i > 0) {
          ok = all_wait(&odone, (n - 1) & 1);  // P and O are free
          tc_fence_after();
        }
        if (moved && i > 0 && ok) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if (16 * c >= hc) break;
            const uint32_t o_col = lanes + 2 * NQ + c0 + 16 * c;
            float v[16];
            tmem_ld16(o_col, v);
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              sum[c][e] *= s_by[0][c0 + 16 * c + e];
              u[e] = __float_as_uint(v[e] * s_by[1][c0 + 16 * c + e]);
            }
            tmem_st16(o_col, u);
          }
          tmem_wait_st();
        }
        // 2^(log2 vs + m - mv) of a column, for the keys of this half-warp
        for (int c = lane & 15; c < hc; c += 16) {
          const float m = s_m[c0 + c], mv = s_mv[c0 + c];
          s_ratio[warp][sub][c] = ex2_approx_f(fminf((m == -INFINITY ? 0.f : m) + sc.y - (mv == -INFINITY ? 0.f : mv), 126.f));
        }
        __syncwarp();
        // ---- probabilities ----
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (16 * c >= hc) break;
          float v[16];
          tmem_ld16(s_col + 16 * c, v);
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 fac = *reinterpret_cast<const float4*>(&s_fac[c0 + 16 * c + e]);
            const float4 m = *reinterpret_cast<const float4*>(&s_m[c0 + 16 * c + e]);
            const float4 ra = *reinterpret_cast<const float4*>(&s_ratio[warp][sub][16 * c + e]);
            const float f4[4] = {fac.x, fac.y, fac.z, fac.w}, m4[4] = {m.x, m.y, m.z, m.w}, r4[4] = {ra.x, ra.y, ra.z, ra.w};
            float pr[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x = v[e + k] * (sc.x * f4[k]) - (m4[k] == -INFINITY ? 0.f : m4[k]);
              if (mask && (!there || at >= s_lim[c0 + 16 * c + e + k])) x = -INFINITY;
              const float y = ex2_approx_f(x);
              sum[c][e + k] += y;
              pr[k] = y * r4[k];
            }
            pk[e / 2] = pack_f16(pr[0], pr[1]), pk[e / 2 + 1] = pack_f16(pr[2], pr[3]);
          }
          const int col = c0 + 16 * c, u = (col & 63) / 8;
          unsigned char* to = sP + (col >> 6) * (kKeys * 128) + key * 128;
          *reinterpret_cast<uint4*>(to + ((u ^ (key & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          *reinterpret_cast<uint4*>(to + (((u + 1) ^ (key & 7)) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
        fence_proxy_async();
        tc_fence_before();
        if (ok) mbar_arrive(&sfree[n & 1]), mbar_arrive(&pready);
      }

      // ---- the part: outputs over these keys, and log2 of the sums ----
      half_sync(half);  // s_red has been read
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (16 * c >= hc) break;
        float l = half_reduce<true>(sum[c], lane);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (lane < 16) s_red[quad][c0 + 16 * c + lane].x = l;
      }
      half_sync(half);
      const int64_t slot = w.slot(a, blockIdx.x);
      for (int c = quad * 32 + lane; c < hc; c += 128) {
        const int col = c0 + c;
        const float l = (s_red[0][col].x + s_red[1][col].x) + (s_red[2][col].x + s_red[3][col].x);
        // l is 0 where no key is seen, and NaN where a score is
        s_out[col] = kv8_out_factor<MODE>(s_mv[col], s_m[col], l);
        if (col < here) a.lses[slot * a.stride + col] = l == 0.f ? -INFINITY : s_m[col] + log2f(l);
      }
      half_sync(half);
      ok = ok && all_wait(&odone, (n - 1) & 1);
      tc_fence_after();
      // lane d of O is dim 4 (d / 4) + (0 2 1 3)[d % 4]
      const int dim = (key & ~3) | (key & 1) << 1 | (key >> 1 & 1);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (16 * c >= hc || !ok) break;
        float v[16];
        tmem_ld16(lanes + 2 * NQ + c0 + 16 * c, v);
        if (key < DIM) {
          float* to = a.parts + (slot * a.stride + c0 + 16 * c) * DIM + dim;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (c0 + 16 * c + e < here) to[e * DIM] = v[e] * s_out[c0 + 16 * c + e];
        }
      }
      tc_fence_before();  // O has been read: the next piece's products may write it (after P's signal)
      asm volatile("bar.sync 3, 256;\n" ::: "memory");  // every column's values have been read
    }
  } else if (warp < kIssuer) {
    set_regs_down<kConvRegs>();
    // ======================= codes to fp16 =======================
    // a lane takes 16 codes at a time; the two rows of eight neighbouring lanes are
    // chosen so that their loads and their stores each fall on different banks
    const int kv = (warp - kSoftWarps) / kConvWarps, cw = (warp - kSoftWarps) % kConvWarps;
    constexpr int kPer = DIM / 16, kStep = 2048 / DIM;
    const int unit = DIM == 128 ? (lane & 3) | ((lane >> 3) & 1) << 2 : lane & 3;
    const int r8 = DIM == 128 ? (lane >> 4 & 1) * 2 : lane >> 2;
    // 128-byte rows: (0 5) (1 4) (2 7) (3 6), the even warps the first of each two pairs
    const int row0c = DIM == 128 ? (cw / 2) * 8 + (((r8 + (cw & 1)) ^ ((lane >> 2 & 1) ? 5 : 0)))
                                 : cw * 8 + r8;
    const int from0 = DIM == 128 ? row0c * 128 + ((unit ^ (row0c & 7)) << 4)
                                 : row0c * 64 + ((unit ^ (row0c >> 1 & 3)) << 4);
    const uint32_t to0 = unit_at(row0c, 2 * unit, kKeys), to1 = unit_at(row0c, 2 * unit + 1, kKeys);
    bool ok = true;
    const uint32_t all = (uint32_t)w.left;
    for (uint32_t n = 0; n < all && ok; ++n) {
      const uint32_t b = n & 1;
      ok = wait(&cfull[kv][b], (n >> 1) & 1);
      if (!ok) break;
      unsigned char* to = smem + (2 * kv + b) * R::tile;
      const unsigned char* from = smem + R::codes_at(kv, b);
      // four rows' codes at a time (rows kStep apart: the swizzle is the same)
#pragma unroll
      for (int e0 = 0; e0 < kPer; e0 += 4) {
        uint4 u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[e] = *reinterpret_cast<const uint4*>(from + from0 + (e0 + e) * kStep * DIM);
        __syncwarp();  // the rows' lanes have read them: half of a row is written over
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 lo, hi;
          kv8_half2<MODE>(u[e].x, lo.x, lo.y);
          kv8_half2<MODE>(u[e].y, lo.z, lo.w);
          kv8_half2<MODE>(u[e].z, hi.x, hi.y);
          kv8_half2<MODE>(u[e].w, hi.z, hi.w);
          *reinterpret_cast<uint4*>(to + to0 + (e0 + e) * kStep * 128) = lo;
          *reinterpret_cast<uint4*>(to + to1 + (e0 + e) * kStep * 128) = hi;
        }
      }
      fence_proxy_async();
      mbar_arrive(kv ? &vfull[b] : &kfull[b]);
    }
  } else {
    set_regs_down<kRestRegs>();
  }
  if (warp == kLoader) {
    // ======================= codes by TMA =======================
    const int boxes = kKeys >> p.shift;
    uint32_t n = 0, issued[2] = {0, 0};
    bool ok = true;
    for (; w.left > 0 && ok; w.next(a)) {
      const int nt = w.count(), h = w.hq / a.blocks;
      const int32_t* pages = p.table + w.g * a.beams * p.cols;
      // page ids and scales are asked for a tile before
      auto page_of = [&](int i) {
        const int64_t j = (int64_t)(w.t + i) * kKeys + (lane << p.shift);
        return lane < boxes && i < nt && j < w.common ? pages[j >> p.shift] : -1;
      };
      auto scale_of = [&](int id) {
        if (id < 0 || id >= p.pages) return make_float2(0.f, 0.f);
        const int64_t tile = (int64_t)id * p.heads + h;
        return make_float2(p.scales[tile], p.scales[tile + p.pages * p.heads]);
      };
      int id = page_of(0), id1 = page_of(1);
      float2 sc = scale_of(id);
      for (int i = 0; i < nt; ++i, ++n) {
        const uint32_t b = n & 1;
        const bool have = id >= 0 && id < p.pages;
        // 16 keys c lie in page c >> (log2 of 16ths of a page)
        const int from = (lane * 16) >> p.shift;
        const float ks = __shfl_sync(0xffffffffu, sc.x, from & 31);
        const float vs = __shfl_sync(0xffffffffu, sc.y, from & 31);
        const bool there = __shfl_sync(0xffffffffu, (int)have, from & 31);
        const unsigned bits = __ballot_sync(0xffffffffu, there && lane < 8);
        const unsigned bytes = __popc(__ballot_sync(0xffffffffu, have)) * (DIM << p.shift);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && all_wait(kv ? &vfree[b] : &kfree[b], ((n >> 1) & 1) ^ 1);
          if (!ok) break;
          if (kv == 0) {
            if (lane < 8) {
              const float2 m = there ? kv8_scales(ks, vs) : make_float2(0.f, -INFINITY);
              meta[n & 3][lane] = make_float2(m.x * kRoot<MODE>, m.y);
            }
            if (lane == 0) valid[n & 3] = (int)bits;
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(&cfull[kv][b], bytes);
          __syncwarp();
          issued[kv] = n + 1;
          if (have)
            tma_load_3d(smem + R::codes_at(kv, b) + (lane << p.shift) * DIM, &a.map, 0, 0,
                        (int)((kv * p.pages + id) * p.heads + h), &cfull[kv][b]);
        }
        if (!ok) break;
        id = id1;
        sc = scale_of(id);
        id1 = page_of(i + 2);
      }
    }
    // no copy is in flight when the CTA ends, whatever ended the loop
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      for (uint32_t i = issued[kv] > 2 ? issued[kv] - 2 : 0; i < issued[kv]; ++i) mbar_wait(&cfull[kv][i & 1], (i >> 1) & 1);
  } else if (warp == kIssuer) {
    // ======================= products =======================
    // Q K^T of a tile goes before P V of the one before it, so that the keys' threads have their
    // next scores while the tensor cores do the outputs.  The whole warp goes through this; one
    // elected lane issues.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    const uint32_t dk = desc_lo(base + R::k, 16), dq = desc_lo(base + R::q, 16), dp = desc_lo(base + R::pt, kKeys * 128);
    const bool lead = elect_one();
    bool ok = true;
    auto qk = [&](uint32_t n) {
      const uint32_t b = n & 1;
      ok = ok && all_wait(&kfull[b], (n >> 1) & 1) && all_wait(&sfree[b], ((n >> 1) & 1) ^ 1);
      if (!ok) return;
      tc_fence_after();
      if (lead) {
#pragma unroll
        for (int s = 0; s < DIM / 16; ++s)
          umma_ss(tm + b * NQ, dk + b * (R::tile >> 4) + (s / 4 * (kKeys * 128) >> 4) + (s % 4) * 2,
                  dq + (s / 4 * (NQ * 128) >> 4) + (s % 4) * 2, kIdQK, s > 0);
        umma_commit(&sfull[b]);
        umma_commit(&kfree[b]);
      }
      __syncwarp();
    };
    uint32_t n = 0, pieces = 0;
    for (; w.left > 0 && ok; w.next(a), ++pieces) {
      const int nt = w.count();
      ok = all_wait(&qready, pieces & 1);
      qk(n);
      for (int i = 0; i < nt && ok; ++i, ++n) {
        if (i + 1 < nt) qk(n + 1);
        const uint32_t b = n & 1;
        ok = ok && all_wait(&pready, n & 1) && all_wait(&vfull[b], (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        // rows 64 and up of V^T: the other panel, or zeros
        const uint32_t dv = desc_lo(base + R::v + b * R::tile, DIM == 128 ? kKeys * 128 : R::zero - R::v - b * R::tile);
        if (lead) {
#pragma unroll
          for (int s = 0; s < kKeys / 16; ++s)
            umma_ss(tm + 2 * NQ, dv + s * (2048 >> 4), dp + s * (2048 >> 4), kIdPV, i > 0 || s > 0);
          umma_commit(&odone);
          umma_commit(&vfree[b]);
        }
        __syncwarp();
      }
    }
    if (n > 0) wait(&odone, (n - 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && abort_flag) atomicOr(&g_kv8_shared_error, 1);
  if (warp == 0) tmem_dealloc(tmem, kCols);
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
  const int64_t grp = r / a.beams;
  const int common = common_of(a, grp), from = min(common, most);
  const int32_t* pages = p.table + r * p.cols;
  const int per = p.heads * a.blocks, tiles = tiles_of(common);  // of the group's tokens
  const int64_t before = tiles_before(a, grp, lane) * per;
  const Shares shares(tiles_before(a, p.rows / a.beams, lane) * per, a.grid);

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
    rowfac[e] = back * p.scale * kLog2eF * kRoot<MODE>;
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

  // ---- keys ----
  const int t0 = from / kTile, t1 = most > from ? (most + kTile - 1) / kTile : t0;
  for (int tile = t0 + warp; tile < t1; tile += kWarps) {
    const int j0 = tile * kTile;
    int64_t block[2];
    bool have[2];
    float ks[2], lv[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int j = j0 + 16 * f;
      const int id = j < most && (j >> p.shift) < p.cols ? pages[j >> p.shift] : -1;
      have[f] = id >= 0 && id < p.pages;
      block[f] = (int64_t)(have[f] ? id : 0) * p.heads + h;
      ks[f] = 0.f, lv[f] = -INFINITY;
      if (have[f]) {
        const float2 sc = kv8_scales(p.scales[block[f]], p.scales[block[f] + p.pages * p.heads]);
        ks[f] = sc.x * kRoot<MODE>, lv[f] = sc.y;
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
            if (at < from || at >= most || at >= end[e] || !have[f]) y = -INFINITY;
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
  grid_dep_wait();  // the parts of the group's tokens
  for (int i = warp; i < rows; i += kWarps) {
    // this row's parts: those of the CTAs whose shares meet its (group, head, block)
    const int qi = (int)(r - grp * a.beams) * (p.tokens * p.group) + i0 + i, hq = h * a.blocks + qi / a.nq, col = qi % a.nq;
    int64_t c0 = 0;
    int n = 0;
    if (tiles > 0) {
      const int64_t u0 = before + (int64_t)hq * tiles;
      c0 = shares.cta_of(u0), n = (int)(shares.cta_of(u0 + tiles - 1) - c0) + 1;
    }
    const int64_t slot = (grp * per + hq + c0) * a.stride + col;  // and every a.stride from there
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = max_nan(top, s_lse[w][i]);
    for (int k = lane; k < n; k += 32) top = max_nan(top, a.lses[slot + (int64_t)k * a.stride]);
    for (int d = 16; d; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    auto add = [&](float c, float4 x) {
      l += c;
      o.x = fmaf(c, x.x, o.x), o.y = fmaf(c, x.y, o.y), o.z = fmaf(c, x.z, o.z), o.w = fmaf(c, x.w, o.w);
    };
    if (top != -INFINITY) {
      for (int w = 0; w < kWarps; ++w)
        add(ex2_approx_f(s_lse[w][i] - top), lane < DIM / 4 ? *reinterpret_cast<const float4*>(&s_o[w][i][4 * lane]) : o);
      // four parts at a time, so that their loads are in flight together
      for (int k0 = 0; k0 < n; k0 += 4) {
        float c[4];
        float4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t at = slot + (int64_t)min(k0 + k, n - 1) * a.stride;
          c[k] = k0 + k < n ? a.lses[at] : -INFINITY;
          x[k] = lane < DIM / 4 ? *reinterpret_cast<const float4*>(a.parts + at * DIM + 4 * lane) : o;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) add(ex2_approx_f(c[k] - top), x[k]);
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

int blocks_of(int64_t rows, int nq) { return (int)((rows + nq - 1) / nq); }

// Sizes that both launches go by.
SharedArgs sized(const Kv8Params& p, int beams) {
  SharedArgs a = {};
  a.p = p;
  a.beams = beams;
  const int64_t rows = (int64_t)beams * p.tokens * p.group;
  a.nq = rows <= 64 ? 64 : 128;
  a.blocks = blocks_of(rows, a.nq);
  a.stride = (int)(rows < a.nq ? rows : a.nq);
  const int64_t tiles = ((int64_t)p.cols * p.page + kKeys - 1) / kKeys * (p.rows / beams) * p.heads * a.blocks;
  a.grid = (int)(tiles < 152 ? tiles : 152);
  return a;
}
// Parts: one for each (group, head, block), and one more for each CTA.
int64_t slots_of(const SharedArgs& a) { return a.p.rows / a.beams * a.p.heads * a.blocks + a.grid; }

template <int MODE, int DIM, int NQ>
gdn_status run_common(const SharedArgs& a, cudaStream_t st) {
  auto kern = kv8_common_kernel<MODE, DIM, NQ>;
  constexpr int bytes = Room<DIM, NQ>::bytes;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return GDN_ERR_CUDA;
  kern<<<a.grid, kThreads, bytes, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int MODE, int DIM>
gdn_status run(SharedArgs& a, cudaStream_t st) {
  const Kv8Params& p = a.p;
  const int64_t rows = (int64_t)p.tokens * p.group;
  const bool few = rows <= 8;
  const int64_t y = few ? 1 : (rows + 15) / 16;
  if (y > 65535) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (p.pages > 0 && !make_map_3d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, DIM, p.page,
                                  (uint64_t)(2 * p.pages * p.heads), DIM, DIM, p.page,
                                  DIM == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return GDN_ERR_CUDA;
  if (a.grid > 0) {
    const gdn_status s = a.nq == 64 ? run_common<MODE, DIM, 64>(a, st) : run_common<MODE, DIM, 128>(a, st);
    if (s != GDN_OK) return s;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * p.heads), (unsigned)y);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = a.grid > 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, kv8_own_kernel<MODE, DIM, 8>, a)
                            : cudaLaunchKernelEx(&cfg, kv8_own_kernel<MODE, DIM, 16>, a);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

size_t kv8_shared_workspace(const Kv8Params& p, int beams, int dim) {
  const SharedArgs a = sized(p, beams);
  return a.grid == 0 ? 0 : (size_t)slots_of(a) * a.stride * (dim + 1) * sizeof(float);
}

gdn_status launch_kv8_shared(const Kv8Params& p, int beams, const int32_t* shared, int mode, int dim,
                             void* workspace, cudaStream_t st) {
  SharedArgs a = sized(p, beams);
  if ((int64_t)p.heads * a.blocks > 1 << 30) return GDN_ERR_UNSUPPORTED_SHAPE;
  a.shared = shared;
  a.parts = static_cast<float*>(workspace);
  a.lses = a.parts + slots_of(a) * a.stride * dim;
  if (mode == GDN_QDQ_E4M3) return dim == 128 ? run<GDN_QDQ_E4M3, 128>(a, st) : run<GDN_QDQ_E4M3, 64>(a, st);
  return dim == 128 ? run<GDN_QDQ_INT8, 128>(a, st) : run<GDN_QDQ_INT8, 64>(a, st);
}

int kv8_shared_device_error(bool reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv8_shared_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_kv8_shared_error, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace gdn
