// Attention over the 8-bit paged cache where the rows of a group have their first tokens in
// common.  Two launches: the group's tokens, once for all its rows, on the tensor cores; then
// each row's own tokens, and the join of both.
//
// The group's tokens.  The query rows of a (group, K/V head) are its rows times their
// queries times the query heads that share the head; they are few, so the products are laid
// out with the keys as the long side.  Per 128 keys and up to 64 query rows:
//     S = K Q^T      (tcgen05, E4M3 or fp16 -> fp32 in TMEM: lane = key, column = query)
//     P = 2^(s - reference), fp16 to shared memory
//     O += V^T P     (lane = dim, column = query)
// and only the columns in use (16, 32 or 64) cost exponentials.  All tiles of all (group, head,
// block of query rows) form one line, of which every CTA takes an equal, contiguous share; what it
// has of a (group, head, block) is a part: outputs over its own keys, and their log-sum-exp.
// A warp brings the codes of K by TMA (a box per page) and one those of V, into rings of their
// own; four turn V's into fp16 and, with INT8 codes, four K's; one lane of a warp issues Q K^T,
// one of another P V; and eight warps are the keys: a thread has one key, and 16 or 32 of the
// queries.  E4M3 codes of K are an operand as they are, q being the sum of two 8-bit numbers.
//
// A score is taken against its column's references (the largest s, and s + log2 of V's scale,
// which is one for 16 lanes) as they are.  Where P, which fp16 has to hold, outgrows them by 2^8, where the
// second has been missing (V scales of 0 give none), or where V's scale is so small that a score outgrows the
// first by 2^60 unseen, the columns concerned get new ones from their maxima and the tile is done
// again.  Each column decides for itself, so a row's result does not depend on the rows beside it; nor on
// its place, where a group's query rows of a K/V head fit one block of 64.  (Blocks lie at different places of
// the line, where CTAs' shares cut their keys differently.)
//
// A row's own tokens.  A CTA takes 8 (or 16) query rows of a (row, K/V head): its warps go through
// 16 keys at a time from registers, again with the keys, and the dims, as the long side of
// warp products, and their parts are joined with those of the group's tokens.  Codes go from global
// memory into the lanes that need them: a score is a sum over dims in any order, so a lane's 16
// bytes of a key are steps of a product whose other operand, q, is laid out alike; and the rows of
// V^T P are dims in any order, so a lane's bytes of each of four keys are its rows of eight
// products, after an exchange of bytes between neighbouring keys.
//
// Measured on a GB300 (both launches, replayed): 16 x 8 beams behind 1096 .. 4096 tokens with 90 .. 150
// of their own, 8 K/V heads of 128, four query heads each, E4M3, 132 MB: 63 us (kv8_attention 148);
// 64 rows behind 16384 with 24 .. 1024 of their own, 102 MB: 92 us (344); 8 beams behind 131072 tokens,
// 4 heads, INT8, 135 MB: 62 us (188); 4 beams behind 1472: 11.6 us (16.5).  Where little is in common
// both launches cost more than they save: 5 x 3 beams of five drafts, 4 MB, 28 us (19).  So do a few rows
// with many tokens of their own, which one CTA goes through for each row and K/V head: 4 rows x 4 heads with
// 8000 behind 1024 take 177 us (21), with 2000 27 (17), with 500 12 (14).
//
// DRAM is at 30 % in the first launch, issue at 38 %.  What bounds it is the chain of a tile from S by P
// to the next.  In the first case 30 to 37 of a keys' warp's 65 to 73 thousand cycles are its own, 1500 to 1850
// for each of 20 tiles; 12 go by before its first scores, 11 to 13 in waits for S, and as many in waits for the
// product of the tile before, since a set has one buffer of P.  In the second (64 columns) 63 of 102 are its
// own, 2350 a tile, in the third 56 to 60 of 93.  A tile that is done again takes about half as long again:
// where V's scale is 0 throughout, 64 rows behind 16384 tokens 102 us beside 67, for a tenth of the pages 75.
// Earlier forms differ from the present one in more than what is named here.  One of 80 us in the first
// case and 70 in the third with parts of the work left out took in the third: without conversions 53, without the
// softmax 59, without both 44, and without loads and products as well 30.  Four units of warps instead of two,
// with 80 registers a thread, spilled and missed the instruction cache 131 times a tile (46 with two then, 51
// now): 80, 129 and 78.  Two that take whole tiles of 32 columns in turn: 69, 104 and 68.  Warp products from rings in
// shared memory instead of tcgen05, for up to 32 rows: 133 and 124 in the first and the third.
// A row's own tokens took 9 us of the first case and 23 of the second behind the first launch (latency; alone 30
// and 31 with cold caches; products that had the queries as the long side, half of each empty, 31 and 32).
#include <cuda.h>

#include <atomic>

#include "kv8_tc.cuh"
#include "launch.h"

namespace gdn {

namespace {

__device__ int g_kv8_shared_error;

constexpr int kWarps = 4;   // own tokens: warps of a CTA
constexpr int kKeys = 128;  // the group's tokens: keys of a tile

// The first kernel: CW query rows (columns) of a block, N of a product.  Two units of four warps
// have 16 (or 32) columns of a tile each, so that what they go through per tile is short, or
// take tiles in turn: `sets` tiles are worked on at a time.  Warps turn codes into fp16: four do V's,
// and with INT8 codes four more K's.
template <int MODE, int CW>
struct Plan {
  static constexpr bool f8 = MODE == GDN_QDQ_E4M3;
  static constexpr int units = 2, soft = 4 * units, conv = f8 ? 4 : 8;
  static constexpr int issue_qk = soft + conv, issue_pv = issue_qk + 1, load_k = issue_qk + 2, load_v = issue_qk + 3;
  static constexpr int threads = (soft + conv + 4) * 32;
  // registers per thread of the warpgroups: together no more than the launch gave
  static constexpr int launch_regs = f8 ? 128 : 96, soft_regs = f8 ? 192 : 144, conv_regs = 64, rest_regs = 64;
  static_assert(units * soft_regs + conv / 4 * conv_regs + rest_regs <= threads / 128 * launch_regs, "register shares");
  static_assert(threads * launch_regs <= 65536, "registers");
  static constexpr int chunks = CW == 64 ? 2 : 1, cols_of = 16 * chunks;  // 16 columns, of a unit
  static constexpr int per_tile = CW / cols_of, sets = units / per_tile, n = CW < 32 ? 32 : CW;
  static constexpr int s_cols = 2 * sets * n;  // S: two of each set; then O, one of each
  static constexpr uint32_t cols = s_cols + sets * n > 128 ? 256 : 128;
};

struct SharedArgs {
  Kv8Params p;
  CUtensorMap map;  // codes, a page of a head per box
  const int32_t* shared;
  float *parts, *lses;  // [slot][stride][DIM], [slot][stride]
  int beams, cw, blocks;  // query rows of a block; blocks of a (group, head)
  int stride;             // query rows of a part
  int grid;               // CTAs of the first launch
};

// Keys of query i of a row (all of them, of the whole row): [0, end).
__device__ __forceinline__ int seen_end(const Kv8Params& p, int64_t len, int i) {
  const int64_t pos = len - p.tokens + i;
  const int64_t most = (int64_t)p.cols * p.page;
  const int all = kv8_clamp(len, 0, most);
  return p.causal ? kv8_clamp(pos + 1, 0, all) : pos < 0 ? 0 : all;
}

// Tokens that a group has in common (those that its first row has), and their tiles.
__device__ __forceinline__ int common_of(const SharedArgs& a, int64_t g) {
  return kv8_clamp(min(a.shared[g], a.p.lengths[g * a.beams]), 0, (int64_t)a.p.cols * a.p.page);
}
__device__ __forceinline__ int tiles_of(int keys) { return (int)(((uint32_t)keys + kKeys - 1) / kKeys); }

// Tiles of the groups before g1, and of all of them, counted for one (head, block).
__device__ __forceinline__ void tiles_before(const SharedArgs& a, int64_t g1, int lane, int64_t& before, int64_t& all) {
  const int64_t groups = a.p.rows / (uint32_t)a.beams;
  before = all = 0;
  for (int64_t g = lane; g < groups; g += 32) {
    const int n = tiles_of(common_of(a, g));
    all += n;
    if (g < g1) before += n;
  }
  for (int d = 16; d; d >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, d);
    all += __shfl_xor_sync(0xffffffffu, all, d);
  }
}

// a / b of numbers >= 0; nearly always both have 32 bits, whose division is far shorter
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Equal shares of the line of `all` tiles: the first `rest` of n CTAs have one tile more.
struct Shares {
  int64_t each, rest, n;
  __device__ __forceinline__ Shares(int64_t all, int grid) {
    n = all < grid ? all : grid;
    each = n > 0 ? quotient(all, n) : 0, rest = all - each * n;
  }
  __device__ __forceinline__ int64_t start(int64_t c) const { return each * c + (c < rest ? c : rest); }
  __device__ __forceinline__ int64_t cta_of(int64_t u) const {
    const int64_t longer = rest * (each + 1);
    return u < longer ? quotient(u, each + 1) : rest + quotient(u - longer, each);
  }
};

// A CTA's way through its share: pieces of (group, head, block).
struct Walk {
  int64_t left, g;
  int common, tiles, hq, t;  // of the group; head * blocks + block; tile
  __device__ __forceinline__ Walk(const SharedArgs& a, int64_t cta, int lane) {
    const int64_t groups = a.p.rows / (uint32_t)a.beams, per = (int64_t)a.p.heads * a.blocks;
    // (32 groups lie in the lanes: nearly always all)
    const int mine = lane < groups ? common_of(a, lane) : 0;
    int64_t before, all = tiles_of(mine);
    if (groups <= 32) {
      for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    } else {
      tiles_before(a, 0, lane, before, all);
    }
    const Shares s(all * per, a.grid);
    left = 0, g = 0, common = tiles = hq = t = 0;
    if (cta >= s.n) return;
    const int64_t u = s.start(cta);
    left = s.start(cta + 1) - u;
    before = 0;
    for (int64_t g0 = 0;; g0 += 32) {
      const int have = g0 == 0 ? mine : g0 + lane < groups ? common_of(a, g0 + lane) : 0;
      int64_t x = tiles_of(have) * per;
      const int64_t here = x;
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + x > u);
      if (hit) {
        const int at = __ffs(hit) - 1;
        g = g0 + at;
        before += __shfl_sync(0xffffffffu, x - here, at);
        common = __shfl_sync(0xffffffffu, have, at);
        break;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    tiles = tiles_of(common);
    const int64_t in = u - before;
    hq = (int)quotient(in, tiles), t = (int)(in - (int64_t)hq * tiles);
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
    const int64_t groups = a.p.rows / (uint32_t)a.beams;
    for (tiles = 0; tiles == 0 && ++g < groups;) common = common_of(a, g), tiles = tiles_of(common);
    if (tiles == 0) left = 0;
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

// Barriers of a unit's four warps, and of all units'.
__device__ __forceinline__ void unit_sync(int unit) {
  asm volatile("bar.sync %0, 128;\n" ::"r"(1 + unit) : "memory");
}
// the same, and whether any of the threads says yes
__device__ __forceinline__ bool unit_any(int unit, bool yes) {
  uint32_t any;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(any)
               : "r"((uint32_t)yes), "r"(1 + unit)
               : "memory");
  return any;
}
template <int THREADS>
__device__ __forceinline__ void units_sync() {
  asm volatile("bar.sync 7, %0;\n" ::"n"(THREADS) : "memory");
}

// O += V^T P: V in rows of 128 bytes, P in rows of 2 N bytes (64: 64-byte swizzle, SBO 512).
template <int N>
__device__ __forceinline__ void umma_pv(uint32_t d, uint32_t v, uint32_t p, uint32_t id, bool acc) {
  constexpr uint32_t hi = N == 64 ? kDescHi : (512u >> 4) | 1u << 14 | 4u << 29;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %5};\n"
      " setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(v), "r"(p), "r"(id), "r"(kDescHi), "r"(hi), "r"((uint32_t)acc));
}

// A place in a ring of N buffers, and the parity of its turn.
template <int N>
struct Ring {
  uint32_t at = 0, turn = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) at = 0, turn ^= 1;
  }
};

// Shared memory of the first kernel: codes of K and of V as they arrive, as many tiles of them as
// there is room for, since what is on its way is what DRAM's latency leaves; fp16 tiles of V and
// (INT8; E4M3 codes are an operand as they are) of K; the queries, and the sets' P.
// V with 64 dims has a panel of zeros for the other 64 lanes of O.
template <int MODE, int DIM, int CW>
struct Room {
  using L = Plan<MODE, CW>;
  static constexpr bool f8 = MODE == GDN_QDQ_E4M3;
  static constexpr int raw = kKeys * DIM, tile = 2 * raw, ptile = kKeys * L::n * 2;
  static constexpr int raws = f8 ? (CW == 64 ? 3 : 4) : 2, vtiles = 2, ktiles = f8 ? 0 : CW == 64 ? 1 : 2;
  static constexpr int k = 0, v = raws * raw, vt = v + raws * raw, zero = vt + vtiles * tile;
  static constexpr int kt = zero + (DIM == 64 ? kKeys * 128 : 0), q = kt + ktiles * tile, pt = q + L::n * DIM * 2;
  static constexpr int bytes = pt + L::sets * ptile + 1024;
  static_assert(bytes <= 227 * 1024 - 10 * 1024, "shared memory (with what the kernel has besides)");
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __half2 c = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&c);
}
// Two E4M3 numbers (the low 16 bits) as fp16.
__device__ __forceinline__ uint32_t half2_of(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return (uint32_t)h.x | (uint32_t)h.y << 16;
}
// The same of V, where bytes that are no number become 448, the largest.  Such bytes stand where no token
// is, and in blocks whose scale is no number, whose keys have a weight of 0 (and not of NaN) for the
// queries that do not see them: 0 times any number is 0.
__device__ __forceinline__ uint32_t v_half2_of(uint32_t codes) {
  const uint32_t x = half2_of(codes);
  const __half2 y = __hmin2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x5f00)));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Where V's scale, against its reference, is below this P does not tell whether a score outgrows its own, and the
// exponential has to: above it one of 2^60 gives a P of 2^8 at least.  So the sums, of less than 2^31 keys, stay below 2^100.
constexpr float kLittle = 0x1p-52f;

template <int MODE, int DIM, int CW>
__global__ void __launch_bounds__(Plan<MODE, CW>::threads, 1) kv8_common_kernel(const __grid_constant__ SharedArgs a) {
  using R = Room<MODE, DIM, CW>;
  using L = Plan<MODE, CW>;
  constexpr bool F8 = R::f8;
  constexpr int G = L::sets, N = L::n, UC = L::cols_of, KC = L::chunks;
  constexpr uint32_t kIdQK = idesc_f16(128, N, 0, 0), kIdPV = idesc_f16(128, N, 1, 1);
  constexpr uint32_t kBE5M2 = 1u << 10;
  constexpr int kKTiles = F8 ? 1 : R::ktiles;
  extern __shared__ unsigned char smem_raw[];
  // codes there, and free; fp16 tiles there, and free; by buffer
  __shared__ __align__(8) uint64_t kin[R::raws], kout[R::raws], vin[R::raws], vout[R::raws];
  __shared__ __align__(8) uint64_t kfull[kKTiles], kfree[kKTiles], vfull[R::vtiles], vfree[R::vtiles];
  __shared__ __align__(8) uint64_t sfull[2 * G], sfree[2 * G], pready[G], odone[G], qready;  // of S by buffer, by set
  __shared__ float2 meta[16][8];  // [tile]: per 16 keys K scale, log2 of V scale
  __shared__ int valid[16];       // bit c: they have a page
  __shared__ __align__(16) int s_lim[CW];    // keys that a column sees
  __shared__ __align__(16) float s_fac[CW];  // factor of a column's scores
  // of a unit's column: references of s and of s + log2 of V's scale; -m; sum; factor of its
  // output; what a move makes of its sums, and of O
  __shared__ __align__(16) float s_m[L::units][UC], s_mv[L::units][UC], s_neg[L::units][UC], s_sum[L::units][UC], s_out[L::units][UC];
  __shared__ __align__(16) float s_by[L::units][2][UC];
  // for 16 keys of a tile: factor of the scores, 2^(log2 vs + m - mv)
  __shared__ __align__(16) float s_by_k[L::soft][2][UC], s_ratio[L::soft][2][UC];
  __shared__ float2 s_red[L::units][4][UC];
  __shared__ uint32_t s_over[L::units][4];  // columns of which a P is too large, by warp
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);  // uniform
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);

  grid_dep_launch();  // the rows' own tokens need nothing of this launch until their join
  if (warp == 0) tmem_alloc(&tmem_slot, L::cols);
  if (tid == 32) {
    for (int i = 0; i < R::raws; ++i) {
      mbar_init(&kin[i], 1), mbar_init(&vin[i], 1);
      mbar_init(&kout[i], F8 ? 1 : 4), mbar_init(&vout[i], 4);
    }
    for (int i = 0; i < R::vtiles; ++i) mbar_init(&vfull[i], 4), mbar_init(&vfree[i], 1);
    for (int i = 0; i < kKTiles; ++i) mbar_init(&kfull[i], 4), mbar_init(&kfree[i], 1);
    for (int i = 0; i < 2 * G; ++i) mbar_init(&sfull[i], 1), mbar_init(&sfree[i], 4 * L::per_tile);
    for (int i = 0; i < G; ++i) mbar_init(&pready[i], 4 * L::per_tile), mbar_init(&odone[i], 1);
    mbar_init(&qready, L::soft);
    abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (DIM == 64) {
    for (int i = tid; i < kKeys * 8; i += L::threads) reinterpret_cast<uint4*>(smem + R::zero)[i] = make_uint4(0, 0, 0, 0);
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
  // one arrival for a warp, whose lanes have all come here
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp < L::soft) {
    set_regs_up<L::soft_regs>();
    // ======================= keys =======================
    // A thread has a key, and its unit's columns of the set's tiles.
    const int unit = warp / 4, quad = warp & 3, key = quad * 32 + lane, half = lane >> 4, l16 = lane & 15;
    const int set = unit / L::per_tile, c0 = unit % L::per_tile * UC;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + c0, o_col = lanes + L::s_cols + set * N;
    unsigned char *sQ = smem + R::q, *sP = smem + R::pt + set * R::ptile + key * (2 * N);
    const int swap = N == 64 ? key & 7 : key >> 1 & 3, u0 = c0 / 8;
    const int per_row = p.tokens * p.group, all_q = a.beams * per_row;
    float *by_k = s_by_k[warp][half], *ratio = s_ratio[warp][half], *neg = s_neg[unit];
    bool ok = true;
    uint32_t n = 0, mine = 0;  // tiles so far, and this set's
    for (; w.left > 0; w.next(a)) {
      const int nt = w.count(), h = w.hq / a.blocks, q0 = w.hq % a.blocks * CW, here = min(all_q - q0, CW);  // columns in use
      // ---- queries: DIM / 8 lanes to a row ----
      {
        constexpr int kLanes = DIM / 8, kAt = 32 / kLanes, kTimes = (CW + L::soft * kAt - 1) / (L::soft * kAt);
        const int u = lane % kLanes;
        uint4 raws[kTimes];  // (all on their way together)
#pragma unroll
        for (int x = 0; x < kTimes; ++x) {
          const int c = warp * kAt + lane / kLanes + x * L::soft * kAt;
          raws[x] = make_uint4(0, 0, 0, 0);
          if (c < CW) {
            const int i = q0 + c, r_in = i / per_row, x_in = i - r_in * per_row;
            const int64_t r = w.g * a.beams + r_in;
            if (c < here)
              raws[x] = __ldg(reinterpret_cast<const uint4*>(p.x + r * p.x_row + (x_in / p.group) * p.x_token +
                                                             (int64_t)(h * p.group + x_in % p.group) * p.x_head + 8 * u));
            if (u == 0) s_lim[c] = c < here ? min(seen_end(p, p.lengths[r], x_in / p.group), w.common) : 0;
          }
        }
#pragma unroll
        for (int x = 0; x < kTimes; ++x) {
          const int c = warp * kAt + lane / kLanes + x * L::soft * kAt;
          const uint4 raw = raws[x];
          float f[8], most = 0.f;
          bf16x8(raw, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[e]));
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
          float up, back;
          kv8_q_factor<F8 ? 7 : 8>(most, up, back);
          if (c >= CW) break;  // (all rows of a warp's or none)
          if (u == 0) s_fac[c] = back * fabsf(p.scale) * kLog2eF;
          if (p.scale < 0.f) up = -up;
          if constexpr (F8) {  // an E4M3 number and an E5M2 one (kv8.cuh)
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float rest[4];
              hi[e] = kv8_q_first(f + 4 * e, up, rest);
              lo[e] = kv8_e5m2x4(rest);
            }
            unsigned char* to = sQ + (u & 1) * 8 + (DIM == 128 ? unit_at(c, u >> 1, N) : c * 64 + (((u >> 1) ^ (c >> 1 & 3)) << 4));
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to + N * DIM) = make_uint2(lo[0], lo[1]);
          } else {
            *reinterpret_cast<uint4*>(sQ + unit_at(c, u, N)) =
                make_uint4(pack_f16(f[0] * up, f[2] * up), pack_f16(f[1] * up, f[3] * up),
                           pack_f16(f[4] * up, f[6] * up), pack_f16(f[5] * up, f[7] * up));
          }
        }
        fence_proxy_async();
        if (ok) warp_arrive(&qready);
      }
      if (quad == 0 && half == 0) {
        for (int c = l16; c < UC; c += 16) s_m[unit][c] = s_mv[unit][c] = -INFINITY, neg[c] = INFINITY;  // no score yet: any is too large
      }
      units_sync<L::soft * 32>();  // the columns' limits and factors
      float my_fac[KC];  // (of the columns that a lane does for its half-warp)
      int my_lim[KC];
      unsigned least_u = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int col = c0 + 16 * c + l16;
        my_fac[c] = s_fac[col], my_lim[c] = s_lim[col];
        if (col < here) least_u = min(least_u, (unsigned)s_lim[col]);
      }
      const int least = (int)__reduce_min_sync(0xffffffffu, least_u);
      float sum[KC][16];
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[c][e] = 0.f;

      const int first = (int)((set - n) & (G - 1));  // this set's first tile of the piece
      for (int i = first; i < nt; i += G, ++mine) {
        const uint32_t buf = (mine & 1) * G + set;
        ok = ok && all_wait(&sfull[buf], mine >> 1 & 1);
        if (i > first) ok = ok && all_wait(&odone[set], (mine - 1) & 1);  // P and O are free
        if (!ok) {  // a wait gave up: only the barriers that others may stand at
          if (unit_any(unit, false)) unit_sync(unit), unit_sync(unit);
          continue;
        }
        tc_fence_after();
        float y[KC][16];
        const int j0 = (w.t + i) * kKeys, at = j0 + key, slot = (n + i) & 15;
        const float2 sc = meta[slot][key >> 4];
        // columns that see this key
        uint32_t see = 0xffffffffu;
        if (valid[slot] != 255 || j0 + kKeys > least) {
          see = 0;
          if (valid[slot] >> (key >> 4) & 1) {
#pragma unroll
            for (int e = 0; e < UC; e += 4) {
              const int4 x = *reinterpret_cast<const int4*>(&s_lim[c0 + e]);
              see |= (uint32_t)(at < x.x) << e | (uint32_t)(at < x.y) << (e + 1) | (uint32_t)(at < x.z) << (e + 2) | (uint32_t)(at < x.w) << (e + 3);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < KC; ++c) by_k[16 * c + l16] = my_fac[c] * sc.x;
        for (int again = 0;; ++again) {
          // A column that has seen V scales of 0 only has no reference for s + log2 of V's scale, and gets
          // one with the first other scale it sees.  (P would not tell: without a reference it is of any size.)
          uint32_t start = 0;
          bool little = false;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const float mv = s_mv[unit][16 * c + l16], um = neg[16 * c + l16];
            const bool sees = j0 + (key & ~15) < my_lim[c];
            if (mv == -INFINITY && sc.y > -INFINITY && sees) start |= 1u << (16 * c + l16);
            const float by = um == INFINITY ? 1.f : ex2_approx_f(fminf(sc.y - um - (mv == -INFINITY ? 0.f : mv), 126.f));
            ratio[16 * c + l16] = by, little |= by < kLittle && sees;
          }
          __syncwarp();
          // (tiles with such scales are looked at below, which tells who needs what; they are few)
          bool over = start != 0 || (little && (valid[slot] >> (key >> 4) & 1));
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            float v[16];
            tmem_ld16(lanes + buf * N + 16 * c, v);
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&by_k[16 * c + e]);
              const float4 m = *reinterpret_cast<const float4*>(&neg[16 * c + e]);
              const float4 r = *reinterpret_cast<const float4*>(&ratio[16 * c + e]);
              float2 x = fma2(make_float2(v[e], v[e + 1]), make_float2(f.x, f.y), make_float2(m.x, m.y));
              float2 z = fma2(make_float2(v[e + 2], v[e + 3]), make_float2(f.z, f.w), make_float2(m.z, m.w));
              float* yy = y[c] + e;
              yy[0] = ex2_approx_f(x.x), yy[1] = ex2_approx_f(x.y), yy[2] = ex2_approx_f(z.x), yy[3] = ex2_approx_f(z.y);
              if (see != 0xffffffffu) {
                if (!(see >> (16 * c + e) & 1)) yy[0] = 0.f;
                if (!(see >> (16 * c + e + 1) & 1)) yy[1] = 0.f;
                if (!(see >> (16 * c + e + 2) & 1)) yy[2] = 0.f;
                if (!(see >> (16 * c + e + 3) & 1)) yy[3] = 0.f;
              }
              x = mul2(make_float2(yy[0], yy[1]), make_float2(r.x, r.y)), z = mul2(make_float2(yy[2], yy[3]), make_float2(r.z, r.w));
              pk[e / 2] = pack_f16(x.x, x.y), pk[e / 2 + 1] = pack_f16(z.x, z.y);
            }
            *reinterpret_cast<uint4*>(sP + (((u0 + 2 * c) ^ swap) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            *reinterpret_cast<uint4*>(sP + (((u0 + 2 * c + 1) ^ swap) << 4)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
            const uint32_t most = max2(max2(max2(pk[0], pk[1]), max2(pk[2], pk[3])), max2(max2(pk[4], pk[5]), max2(pk[6], pk[7])));
            over |= (most & 0xffffu) > 0x5c00u || most >> 16 > 0x5c00u;  // of numbers >= 0: above 256
          }
          // Does a column need other references?  (fp16 and the sums have the room for 2^8.)  Then it gets
          // them from its maxima, and the tile goes once more; what is too large after that is no number.  Only
          // columns with a need of their own: another's scores may have outgrown theirs where V's scale is
          // small, and would move or not as its neighbours do.
          if (again || !unit_any(unit, over)) break;
          uint32_t too = start;
#pragma unroll
          for (int c = 0; c < KC; ++c) ratio[16 * c + l16] = fmaxf(ratio[16 * c + l16], kLittle);
          __syncwarp();
#pragma unroll
          for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 r = *reinterpret_cast<const float2*>(&ratio[16 * c + e]);
              const float2 x = mul2(make_float2(y[c][e], y[c][e + 1]), r);
              const uint32_t both = pack_f16(x.x, x.y);
              too |= (uint32_t)((both & 0xffffu) > 0x5c00u) << (16 * c + e) | (uint32_t)(both >> 16 > 0x5c00u) << (16 * c + e + 1);
            }
          too = __reduce_or_sync(0xffffffffu, too);
          if (lane == 0) s_over[unit][quad] = too;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            float x[16];
            tmem_ld16(lanes + buf * N + 16 * c, x);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!(see >> (16 * c + e) & 1)) x[e] = -INFINITY;
            const float top = half_reduce<false>(x, lane);
            // (a factor of 0 would make -inf a NaN)
            float nm = top == -INFINITY ? top : top * (my_fac[c] * sc.x);
            float nv = nm + sc.y;
            nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 16));
            nv = fmaxf(nv, __shfl_xor_sync(0xffffffffu, nv, 16));
            if (half == 0) s_red[unit][quad][16 * c + l16] = make_float2(nm, nv);
          }
          unit_sync(unit);
          if (quad == 0) {
            const uint32_t moves = s_over[unit][0] | s_over[unit][1] | s_over[unit][2] | s_over[unit][3];
            for (int c = lane; c < UC; c += 32) {
              float nm = -INFINITY, nv = -INFINITY;
#pragma unroll
              for (int q = 0; q < 4; ++q) nm = fmaxf(nm, s_red[unit][q][c].x), nv = fmaxf(nv, s_red[unit][q][c].y);
              // (scores that are all below fp32's range have a weight of 0, for which the reference has to be a number)
              nm = fmaxf(nm, -3.402823466e38f);
              const float m = s_m[unit][c], mv = s_mv[unit][c];
              float by = 1.f, by_o = 1.f;
              if ((moves >> c & 1) && nm > m + 8.f) by = ex2_approx_f(m - nm), s_m[unit][c] = nm, neg[c] = -nm;
              if ((moves >> c & 1) && nv > mv + 8.f) by_o = ex2_approx_f(mv - nv), s_mv[unit][c] = nv;
              s_by[unit][0][c] = by, s_by[unit][1][c] = by_o;
            }
          }
          unit_sync(unit);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[c][e] *= s_by[unit][0][16 * c + e];
            if (i > first) {
              float o[16];
              tmem_ld16(o_col + 16 * c, o);
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * s_by[unit][1][16 * c + e]);
              tmem_st16(o_col + 16 * c, u);
            }
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 x = add2(make_float2(sum[c][e], sum[c][e + 1]), make_float2(y[c][e], y[c][e + 1]));
            sum[c][e] = x.x, sum[c][e + 1] = x.y;
          }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[set]), mbar_arrive(&sfree[buf]);
      }

      // ---- the part: outputs over the piece's keys, and log2 of the sums ----
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        float l = half_reduce<true>(sum[c], lane);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (half == 0) s_red[unit][quad][16 * c + l16].x = l;
      }
      if (first < nt) {
        ok = ok && all_wait(&odone[set], (mine - 1) & 1);
        tc_fence_after();
      }
      unit_sync(unit);
      if (quad == 0)
        for (int c = lane; c < UC; c += 32)
          s_sum[unit][c] = (s_red[unit][0][c].x + s_red[unit][1][c].x) + (s_red[unit][2][c].x + s_red[unit][3][c].x);
      tc_fence_before();
      units_sync<L::soft * 32>();
      tc_fence_after();
      // the first set's units join the others' to their own
      const int64_t slot = w.slot(a, blockIdx.x);
      if (set == 0) {
        if (quad == 0) {
          for (int c = lane; c < UC; c += 32) {
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int x = 0; x < G; ++x) m = fmaxf(m, s_m[x * L::per_tile + unit][c]);
#pragma unroll
            for (int x = 0; x < G; ++x) {
              const float part = s_sum[x * L::per_tile + unit][c];
              l += m == -INFINITY ? part : part * ex2_approx_f(s_m[x * L::per_tile + unit][c] - m);
            }
            // l is 0 where no key is seen, and NaN where a score is  (V as it is: no power of two is left)
#pragma unroll
            for (int x = 0; x < G; ++x)
              s_out[x * L::per_tile + unit][c] = kv8_out_factor<GDN_QDQ_INT8>(s_mv[x * L::per_tile + unit][c], m, l);
            if (c0 + c < here) a.lses[slot * a.stride + c0 + c] = l == 0.f ? -INFINITY : m + log2f(l);
          }
        }
        unit_sync(unit);
#pragma unroll 1
        for (int c = 0; c < KC && ok; ++c) {
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
#pragma unroll 1
          for (int x = 0; x < G; ++x) {
            if ((int)((x - n) & (G - 1)) >= nt) continue;  // no tile of the piece was this set's
            float v[16];
            tmem_ld16(lanes + L::s_cols + x * N + 16 * c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(v[e], s_out[x * L::per_tile + unit][16 * c + e], o[e]);
          }
          // with INT8 codes lane d of O is dim 4 (d / 4) + (0 2 1 3)[d % 4]
          const int dim = F8 ? key : (key & ~3) | (key & 1) << 1 | (key >> 1 & 1);
          if (key < DIM) {
            float* to = a.parts + (slot * a.stride + c0 + 16 * c) * DIM + dim;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (c0 + 16 * c + e < here) to[e * DIM] = o[e];
          }
        }
      }
      n += nt;
      tc_fence_before();  // O has been read: the next piece's products may write it (after P's signal)
      units_sync<L::soft * 32>();       // every column's values have been read
      tc_fence_after();
    }
  } else if (warp < L::issue_qk) {
    set_regs_down<L::conv_regs>();
    // ======================= codes to fp16 =======================
    // a lane takes 16 codes at a time; the two rows of eight neighbouring lanes are
    // chosen so that their loads and their stores each fall on different banks
    const int cw = (warp - L::soft) % 4, second = (warp - L::soft) / 4;
    constexpr int kPer = DIM / 16, kStep = 2048 / DIM;
    const int unit = DIM == 128 ? (lane & 3) | ((lane >> 3) & 1) << 2 : lane & 3;
    const int r8 = DIM == 128 ? (lane >> 4 & 1) * 2 : lane >> 2;
    // 128-byte rows: (0 5) (1 4) (2 7) (3 6), the even warps the first of each two pairs
    const int row0c = DIM == 128 ? (cw / 2) * 8 + (((r8 + (cw & 1)) ^ ((lane >> 2 & 1) ? 5 : 0)))
                                 : cw * 8 + r8;
    const int from0 = DIM == 128 ? row0c * 128 + ((unit ^ (row0c & 7)) << 4)
                                 : row0c * 64 + ((unit ^ (row0c >> 1 & 3)) << 4);
    const uint32_t to0 = unit_at(row0c, 2 * unit, kKeys), to1 = unit_at(row0c, 2 * unit + 1, kKeys);
    // Tiles of V, or (INT8, the first four warps) of K: the same code, which stays where instructions
    // are near.  (Rows kStep apart: the swizzle is the same.)
    const uint32_t all = (uint32_t)w.left;
    const bool is_k = !F8 && !second;
    for (uint32_t n = 0; n < all; ++n) {
      const uint32_t outs = is_k ? kKTiles : R::vtiles, in = n % R::raws, out = n % outs;
      if (!all_wait((is_k ? kin : vin) + in, n / R::raws & 1)) break;
      const unsigned char* from = smem + (is_k ? R::k : R::v) + in * R::raw + from0;
      unsigned char* to = smem + (is_k ? R::kt : R::vt) + out * R::tile;
      if (!all_wait((is_k ? kfree : vfree) + out, (n / outs & 1) ^ 1)) break;
      constexpr int kAt = 4;
#pragma unroll 1
      for (int e0 = 0; e0 < kPer; e0 += kAt) {
        uint4 u[kAt];
#pragma unroll
        for (int e = 0; e < kAt; ++e) u[e] = *reinterpret_cast<const uint4*>(from + (e0 + e) * kStep * DIM);
#pragma unroll
        for (int e = 0; e < kAt; ++e) {
          uint4 lo, hi;
          if constexpr (F8) {
            lo.x = v_half2_of(u[e].x), lo.y = v_half2_of(u[e].x >> 16), lo.z = v_half2_of(u[e].y), lo.w = v_half2_of(u[e].y >> 16);
            hi.x = v_half2_of(u[e].z), hi.y = v_half2_of(u[e].z >> 16), hi.z = v_half2_of(u[e].w), hi.w = v_half2_of(u[e].w >> 16);
          } else {
            kv8_half2<MODE>(u[e].x, lo.x, lo.y);
            kv8_half2<MODE>(u[e].y, lo.z, lo.w);
            kv8_half2<MODE>(u[e].z, hi.x, hi.y);
            kv8_half2<MODE>(u[e].w, hi.z, hi.w);
          }
          *reinterpret_cast<uint4*>(to + to0 + (e0 + e) * kStep * 128) = lo;
          *reinterpret_cast<uint4*>(to + to1 + (e0 + e) * kStep * 128) = hi;
        }
      }
      warp_arrive((is_k ? kout : vout) + in);
      fence_proxy_async();
      warp_arrive((is_k ? kfull : vfull) + out);
    }
  } else {
    set_regs_down<L::rest_regs>();
  }
  if (warp == L::load_k || warp == L::load_v) {
    // ======================= codes by TMA =======================
    // A warp for K, which says what the tile has, and one for V.
    // Lane l has page l of a window of 32, and its scales; those of the next window are asked for
    // while this one's tiles are loaded.
    const bool is_v = warp == L::load_v;
    const int boxes = kKeys >> p.shift, shift = 31 - __clz(boxes), span = 32 >> shift;  // pages of a tile; tiles of a window
    uint64_t *in = is_v ? vin : kin, *free = is_v ? vout : kout;
    constexpr int bufs = R::raws;
    uint32_t n = 0, issued = 0, b = 0, turn = 0;
    bool ok = true;
    for (; w.left > 0 && ok; w.next(a)) {
      const int nt = w.count(), h = w.hq / a.blocks;
      const int32_t* pages = p.table + w.g * a.beams * p.cols;
      auto page_of = [&](int i) {  // of the window that begins with tile i
        const int64_t j = ((int64_t)(w.t + i) * kKeys) + ((int64_t)lane << p.shift);
        const int id = i + (lane >> shift) < nt && j < w.common ? pages[j >> p.shift] : -1;
        return id < p.pages ? id : -1;
      };
      auto scale_of = [&](int id) {
        if (is_v || id < 0) return make_float2(0.f, 0.f);
        const int64_t tile = (int64_t)id * p.heads + h;
        return make_float2(p.scales[tile], p.scales[tile + p.pages * p.heads]);
      };
      int id = -1, later = page_of(0);
      float2 sc = make_float2(0.f, 0.f), sc_later = scale_of(later);
      for (int i = 0; i < nt; ++i, ++n) {
        const int at = i & (span - 1);  // in the window
        if (at == 0) id = later, sc = sc_later, later = page_of(i + span);
        if (at == 1) sc_later = scale_of(later);
        ok = all_wait(&free[b], turn ^ 1);
        if (!ok) break;
        const bool have = id >= 0, now = lane >> shift == at;
        if (have && now)
          tma_load_3d(smem + (is_v ? R::v : R::k) + b * R::raw + ((lane & (boxes - 1)) << p.shift) * DIM, &a.map, 0, 0,
                      (int)((is_v * p.pages + id) * p.heads + h), &in[b]);
        issued = n + 1;
        if (!is_v) {
          // 16 keys c lie in page c >> (log2 of 16ths of a page) of the tile
          const int from = (at << shift) + ((lane * 16 >> p.shift) & (boxes - 1));
          const float k1 = __shfl_sync(0xffffffffu, sc.x, from), v1 = __shfl_sync(0xffffffffu, sc.y, from);
          const bool there = __shfl_sync(0xffffffffu, (int)have, from);
          const unsigned bits = __ballot_sync(0xffffffffu, there && lane < 8);
          // (this buffer of codes is free, so its last tile is multiplied, or its fp16 form waits for
          // that of the tile before: tiles 16 back have been through everything)
          if (lane < 8) meta[n & 15][lane] = there ? kv8_scales(k1, v1) : make_float2(0.f, -INFINITY);
          if (lane == 0) valid[n & 15] = (int)bits;
        }
        const unsigned bytes = __popc(__ballot_sync(0xffffffffu, have && now)) * (DIM << p.shift);
        __syncwarp();
        if (lane == 0) mbar_expect_tx(&in[b], bytes);
        if (++b == bufs) b = 0, turn ^= 1;
      }
    }
    // no copy is in flight when the CTA ends, whatever ended the loop
    for (uint32_t i = issued > bufs ? issued - bufs : 0; i < issued; ++i) mbar_wait(&in[i % bufs], (i / bufs) & 1);
  } else if (warp == L::issue_qk || warp == L::issue_pv) {
    // ======================= products =======================
    // A warp for Q K^T, one for P V.  Each goes through this as a whole, and what it goes by comes
    // from one lane, so that descriptors stay in uniform registers; one elected lane issues.  (One
    // warp for both, on registers of its lanes, took 1500 cycles for a tile.)
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    const bool lead = elect_one();
    uint32_t left = (uint32_t)__shfl_sync(0xffffffffu, (int)w.left, 0);
    bool ok = true;
    uint32_t n = 0;
    if (warp == L::issue_qk) {
      const uint32_t dk = desc_lo(base + (F8 ? R::k : R::kt), 16), dq = desc_lo(base + R::q, 16);
      Ring<F8 ? R::raws : kKTiles> kb;
      uint64_t *there = F8 ? kin : kfull, *gone = F8 ? kout : kfree;
      for (uint32_t pieces = 0; left > 0 && ok; w.next(a), ++pieces) {
        const uint32_t nt = (uint32_t)__shfl_sync(0xffffffffu, w.count(), 0);
        ok = all_wait(&qready, pieces & 1);
        for (uint32_t i = 0; i < nt; ++i, ++n) {
          const uint32_t buf = (n / G & 1) * G + (n & (G - 1));
          ok = ok && all_wait(&there[kb.at], kb.turn) && all_wait(&sfree[buf], (n / G >> 1 & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          if (lead) {
            const uint32_t d = tm + buf * N, k = dk + kb.at * ((F8 ? R::raw : R::tile) >> 4);
            if constexpr (F8) {
              constexpr int kRow = DIM / 32;
#pragma unroll
              for (int s = 0; s < 2 * kRow; ++s)  // q's first parts, then its second ones, with the same codes
                umma_ss_f8<DIM>(d, k + s % kRow * 2, dq + (s / kRow * (N * DIM) >> 4) + s % kRow * 2, kIdQK | (s < kRow ? 0 : kBE5M2), s > 0);
            } else {
#pragma unroll
              for (int s = 0; s < DIM / 16; ++s)
                umma_ss(d, k + (s / 4 * (kKeys * 128) >> 4) + (s % 4) * 2, dq + (s / 4 * (N * 128) >> 4) + (s % 4) * 2, kIdQK, s > 0);
            }
            umma_commit(&gone[kb.at]);
            umma_commit(&sfull[buf]);  // (the one that is waited for at the end)
          }
          __syncwarp();
          kb.next();
        }
        left -= nt;
      }
    } else {
      const uint32_t dp = desc_lo(base + R::pt, 16);
      Ring<R::vtiles> vb;
      for (; left > 0 && ok; w.next(a)) {
        const uint32_t nt = (uint32_t)__shfl_sync(0xffffffffu, w.count(), 0);
        for (uint32_t i = 0; i < nt; ++i, ++n) {
          const uint32_t g = n & (G - 1);
          ok = ok && all_wait(&vfull[vb.at], vb.turn) && all_wait(&pready[g], n / G & 1);
          if (!ok) break;
          tc_fence_after();
          // rows 64 and up of V^T: the other panel, or zeros
          const uint32_t dv = desc_lo(base + R::vt + vb.at * R::tile, DIM == 128 ? kKeys * 128 : R::zero - R::vt - vb.at * R::tile);
          if (lead) {
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              umma_pv<N>(tm + L::s_cols + g * N, dv + s * (2048 >> 4), dp + g * (R::ptile >> 4) + s * (N * 32 >> 4), kIdPV, i >= G || s > 0);
            umma_commit(&vfree[vb.at]);
            umma_commit(&odone[g]);
          }
          __syncwarp();
          vb.next();
        }
        left -= nt;
      }
    }
    // every product issued has completed before the CTA ends
    if (warp == L::issue_qk) {
      for (uint32_t buf = 0; buf < 2 * G; ++buf) {
        // tiles n with (n / G & 1) * G + (n & (G - 1)) == buf
        const uint32_t uses = (n + 2 * G - 1 - buf) / (2 * G);
        if (uses > 0) wait(&sfull[buf], (uses - 1) & 1);
      }
    } else {
      for (uint32_t g = 0; g < G; ++g) {
        const uint32_t tiles = (n + G - 1 - g) / G;
        if (tiles > 0) wait(&odone[g], (tiles - 1) & 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && abort_flag) atomicOr(&g_kv8_shared_error, 1);
  if (warp == 0) tmem_dealloc(tmem, L::cols);
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

// Transposes 8 x 8 numbers of 16 bits, two of a row in a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}

// Where a lane's codes of a key (step c, word w) lie in the key's dims; lane % 4 == t.
template <int DIM>
__device__ __forceinline__ int dim_of(int t, int c, int w) {
  return (DIM == 128 ? 32 * t + 16 * c : 16 * t) + 4 * w;
}

// 8 NB query rows in a warp, the keys coming 16 at a time: S = K Q^T and O += V^T P as warp
// products with the keys, then the dims, as the long side.  Lane (g, t): scores of keys g and
// g + 8 for queries 2 t and 2 t + 1 of each eight; outputs of these at dims DIM / 8 g ...
template <int MODE, int DIM, int NB>
struct Rows {
  static constexpr int KC = DIM / 64, KS = DIM / 16, MT = DIM / 16;
  static constexpr bool F8 = MODE == GDN_QDQ_E4M3;
  using V = typename Codes<DIM>::T;
  float o[MT][NB][4], l[NB][2], m[NB][2], mv[NB][2], fac[NB][2];
  int lim[NB][2];  // keys that the query sees

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b) o[j][b][0] = o[j][b][1] = o[j][b][2] = o[j][b][3] = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) l[b][e] = 0.f, m[b][e] = mv[b][e] = -INFINITY;
  }
  // Four codes of a key of K, or two of each of two of V, as fp16.
  template <bool OF_V>
  static __device__ __forceinline__ void two(uint32_t w, uint32_t& first, uint32_t& second) {
    if constexpr (!F8) kv8_half2<MODE>(w, first, second);
    else if constexpr (OF_V) first = v_half2_of(w), second = v_half2_of(w >> 16);
    else first = half2_of(w), second = half2_of(w >> 16);
  }
  // The products' other operand: eight queries, of which a lane has row g, by step.
  static __device__ __forceinline__ uint2 query_of(uint2 raw, float to) {
    float f[4];
    bf16x4(raw, f);
    return F8 ? make_uint2(pack_f16(f[0] * to, f[1] * to), pack_f16(f[2] * to, f[3] * to))
              : make_uint2(pack_f16(f[0] * to, f[2] * to), pack_f16(f[1] * to, f[3] * to));
  }

  // 16 keys from position j0: K of keys g and g + 8, V of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9.
  // part: not every query sees all of them, or they are not all of [from, to) or there.
  template <class Q>
  __device__ __forceinline__ void step(const uint4 (&kc)[2][KC], const V (&vc)[4], const Q& query, float ks, float lv,
                                       bool part, int j0, int from, int to, bool there, int g, int t) {
    float s[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const uint32_t x[4] = {kc[0][c].x, kc[0][c].y, kc[0][c].z, kc[0][c].w};
      const uint32_t y[4] = {kc[1][c].x, kc[1][c].y, kc[1][c].z, kc[1][c].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a[4];
        two<false>(x[w], a[0], a[2]);
        two<false>(y[w], a[1], a[3]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint2 q = query(4 * c + w, b);
          mma_f16(s[b], a, q.x, q.y);
        }
      }
    }
    // ---- scores; does one outgrow its query's references by 2^8? ----
    bool over = false;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = fac[b][e] * ks, most = fminf(m[b][e] + 8.f, mv[b][e] + 8.f - lv);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x = s[b][2 * h + e] * f;
          if (part) {
            const int j = j0 + g + 8 * h;
            if (j < from || j >= to || j >= lim[b][e] || !there) x = -INFINITY;
          }
          s[b][2 * h + e] = x;
          over |= x > most;
        }
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float nm = fmaxf(s[b][e], s[b][2 + e]);
          nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 4));
          nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 8));
          nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, 16));
          const float nv = nm + lv;
          if (nm > m[b][e] + 8.f) l[b][e] *= ex2_approx_f(m[b][e] - nm), m[b][e] = nm;
          if (nv > mv[b][e] + 8.f) {
            const float by = ex2_approx_f(mv[b][e] - nv);
            mv[b][e] = nv;
#pragma unroll
            for (int j = 0; j < MT; ++j) o[j][b][e] *= by, o[j][b][2 + e] *= by;
          }
        }
    }
    // ---- probabilities: from (key, queries) to (query, keys) ----
    uint32_t pb[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float y[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float um = m[b][e] == -INFINITY ? 0.f : m[b][e], uv = mv[b][e] == -INFINITY ? 0.f : mv[b][e];
        const float ratio = ex2_approx_f(fminf(um + lv - uv, 126.f));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w = ex2_approx_f(s[b][2 * h + e] - um);
          l[b][e] += w;
          y[2 * h + e] = w * ratio;
        }
      }
      pb[b][0] = transpose8(pack_f16(y[0], y[1]));
      pb[b][1] = transpose8(pack_f16(y[2], y[3]));
    }
    // ---- outputs: rows g and g + 8 of product j are dims 2 j and 2 j + 1 of the lane's ----
    const uint32_t* w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) w[x] = reinterpret_cast<const uint32_t*>(&vc[x]);
#pragma unroll
    for (int i = 0; i < DIM / 32; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        // of two neighbouring keys a, b: a0 b0 a1 b1 (E4M3), a0 a1 b0 b1 (INT8), then those of 2 and 3
        const uint32_t sel = F8 ? (z ? 0x7362 : 0x5140) : (z ? 0x7632 : 0x5410);
        uint32_t a[4];
        two<true>(__byte_perm(w[0][i], w[1][i], sel), a[0], a[1]);
        two<true>(__byte_perm(w[2][i], w[3][i], sel), a[2], a[3]);
#pragma unroll
        for (int b = 0; b < NB; ++b) mma_f16(o[2 * i + z][b], a, pb[b][0], pb[b][1]);
      }
  }

  // Outputs over this warp's keys to to[query][DIM], and log2 of the sums to lse[query].
  __device__ __forceinline__ void finish(float* to, float* lse, int g, int t) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[b][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const float f = kv8_out_factor<GDN_QDQ_INT8>(mv[b][e], m[b][e], x);  // (V as it is)
        const int row = 8 * b + 2 * t + e;
        if (g == 0) lse[row] = x == 0.f ? -INFINITY : m[b][e] + log2f(x);
#pragma unroll
        for (int j = 0; j < MT; j += 2)
          *reinterpret_cast<float4*>(to + row * DIM + DIM / 8 * g + 2 * j) =
              make_float4(o[j][b][e] * f, o[j][b][2 + e] * f, o[j + 1][b][e] * f, o[j + 1][b][2 + e] * f);
      }
  }
};

// The queries of eight rows as operand; row g of this lane is query row i (have: it exists).
// Gives the row's factor of the scores.
template <int MODE, int DIM, class Put>
__device__ __forceinline__ float load_rows(const Kv8Params& p, const __nv_bfloat16* x, bool have, int t, const Put& put) {
  constexpr int KS = DIM / 16;
  uint2 raw[KS];
  float most = 0.f;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    raw[s] = have ? *reinterpret_cast<const uint2*>(x + dim_of<DIM>(t, s / 4, s % 4)) : make_uint2(0, 0);
    float f[4];
    bf16x4(raw[s], f);
    most = fmaxf(most, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
  }
  most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
  float to, back;
  kv8_q_factor<8>(most, to, back);
#pragma unroll
  for (int s = 0; s < KS; ++s) put(s, Rows<MODE, DIM, 1>::query_of(raw[s], to));
  return back * p.scale * kLog2eF;
}

// A row's own tokens, and the join.  ROWS = 8 NB query rows of the CTA.
template <int MODE, int DIM, int NB>
__global__ void __launch_bounds__(kWarps * 32) kv8_own_kernel(const __grid_constant__ SharedArgs a) {
  using R = Rows<MODE, DIM, NB>;
  constexpr int ROWS = 8 * NB;
  __shared__ __align__(16) float s_o[kWarps][ROWS][DIM];
  __shared__ float s_lse[kWarps][ROWS];
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, t = lane % 4;
  const int64_t r = blockIdx.x / p.heads;
  const int h = blockIdx.x % p.heads, i0 = blockIdx.y * ROWS, rows_in = min(p.tokens * p.group - i0, ROWS);
  const int64_t len = p.lengths[r];
  const int most = kv8_clamp(len, 0, (int64_t)p.cols * p.page);
  const int64_t grp = r / a.beams;
  const int common = common_of(a, grp), from = min(common, most);
  const int32_t* pages = p.table + r * p.cols;
  R rows;
  rows.clear();
  uint2 q[R::KS][NB];
  int least = 0x7fffffff;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int i = i0 + 8 * b + g;
    const __nv_bfloat16* x = p.x + r * p.x_row + (i / p.group) * p.x_token + (int64_t)(h * p.group + i % p.group) * p.x_head;
    const float f = load_rows<MODE, DIM>(p, x, 8 * b + g < rows_in, t, [&](int s, uint2 y) { q[s][b] = y; });
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = 8 * b + 2 * t + e;
      rows.fac[b][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + e));
      rows.lim[b][e] = c < rows_in ? seen_end(p, len, (i0 + c) / p.group) : 0;
      if (c < rows_in) least = min(least, rows.lim[b][e]);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);

  // ---- keys, 16 at a time; the next ones are on their way ----
  const int t0 = from / 16 + warp, t1 = most > from ? (most + 15) / 16 : 0;
  uint4 kc[2][R::KC];
  typename R::V vc[4];
  float ks = 0.f, vs = 0.f;
  bool there = false;
  int id = -1;
  auto page_of = [&](int tile) { return tile < t1 ? pages[(tile * 16) >> p.shift] : -1; };
  auto load = [&](int tile) {
    there = id >= 0 && id < p.pages;
    const int64_t block = (int64_t)(there ? id : 0) * p.heads + h;
    const int y = tile * 16 & (p.page - 1);
    ks = vs = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < R::KC; ++c) {
        kc[x][c] = make_uint4(0, 0, 0, 0);
        if (there) kc[x][c] = __ldg(reinterpret_cast<const uint4*>(p.codes + (block * p.page + y + g + 8 * x) * DIM + dim_of<DIM>(t, c, 0)));
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      vc[x] = typename R::V();
      if (there)
        vc[x] = __ldg(reinterpret_cast<const typename R::V*>(
            p.codes + ((block + p.pages * p.heads) * p.page + y + 2 * t + (x & 1) + 8 * (x >> 1)) * DIM + DIM / 8 * g));
    }
    if (there) ks = p.scales[block], vs = p.scales[block + p.pages * p.heads];
  };
  id = page_of(t0);
  if (t0 < t1) load(t0);
  id = page_of(t0 + kWarps);
  for (int tile = t0; tile < t1; tile += kWarps) {
    uint4 k[2][R::KC];
    typename R::V v[4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < R::KC; ++c) k[x][c] = kc[x][c];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = vc[x];
    const float2 sc = there ? kv8_scales(ks, vs) : make_float2(0.f, -INFINITY);
    const bool have = there;
    if (tile + kWarps < t1) load(tile + kWarps);
    id = page_of(tile + 2 * kWarps);
    rows.step(k, v, [&](int s, int b) { return q[s][b]; }, sc.x, sc.y, !have || tile * 16 < from || tile * 16 + 16 > least,
              tile * 16, from, most, have, g, t);
  }
  rows.finish(&s_o[warp][0][0], s_lse[warp], g, t);
  // places of the group's parts
  const int per = p.heads * a.blocks, tiles = tiles_of(common);
  int64_t before, all;
  tiles_before(a, grp, lane, before, all);
  before *= per;
  const Shares shares(all * per, a.grid);
  __syncthreads();
  grid_dep_wait();  // the parts of the group's tokens
  // With sixteen rows a warp's four go side by side, so that their loads are in flight together (30
  // (row, head) of 15 rows: 33 us one after the other, 29 so).
  constexpr int kMine = NB == 1 ? 1 : ROWS / kWarps;
#pragma unroll 1
  for (int i1 = warp; i1 < rows_in; i1 += kMine * kWarps) {
    int64_t slot[kMine];  // of the row's first part in the workspace, and every a.stride from there
    int n[kMine], most_n = 0;
    float top[kMine], l[kMine];
    float4 o[kMine];
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      // this row's parts: those of the CTAs whose shares meet its (group, head, block)
      const int i = i1 + x * kWarps;
      const int qi = (int)(r - grp * a.beams) * (p.tokens * p.group) + i0 + i, hq = h * a.blocks + qi / a.cw;
      int64_t c0 = 0;
      n[x] = 0;
      if (tiles > 0 && i < rows_in) {
        const int64_t u0 = before + (int64_t)hq * tiles;
        c0 = shares.cta_of(u0), n[x] = (int)(shares.cta_of(u0 + tiles - 1) - c0) + 1;
      }
      slot[x] = (grp * per + hq + c0) * a.stride + qi % a.cw;
      most_n = max(most_n, n[x]);
      top[x] = -INFINITY, l[x] = 0.f, o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto lse_of = [&](int x, int k) { return k < n[x] ? a.lses[slot[x] + (int64_t)k * a.stride] : -INFINITY; };
    for (int k = lane; k - lane < most_n; k += 32)
#pragma unroll
      for (int x = 0; x < kMine; ++x) top[x] = max_nan(top[x], lse_of(x, k));
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      for (int w = 0; w < kWarps; ++w) top[x] = max_nan(top[x], s_lse[w][i1 + x * kWarps]);
      for (int d = 16; d; d >>= 1) top[x] = max_nan(top[x], __shfl_xor_sync(0xffffffffu, top[x], d));
    }
    // (a weight of 0 for rows without a score)
    auto add = [&](int x, float lse, float4 v) {
      const float c = top[x] == -INFINITY ? 0.f : ex2_approx_f(lse - top[x]);
      l[x] += c;
      o[x].x = fmaf(c, v.x, o[x].x), o[x].y = fmaf(c, v.y, o[x].y), o[x].z = fmaf(c, v.z, o[x].z), o[x].w = fmaf(c, v.w, o[x].w);
    };
    const int at4 = 4 * (lane % (DIM / 4));
#pragma unroll
    for (int x = 0; x < kMine; ++x)
      for (int w = 0; w < kWarps; ++w) add(x, s_lse[w][i1 + x * kWarps], *reinterpret_cast<const float4*>(&s_o[w][i1 + x * kWarps][at4]));
    for (int k0 = 0; k0 < most_n; k0 += 32) {
      float lse[kMine];
#pragma unroll
      for (int x = 0; x < kMine; ++x) lse[x] = lse_of(x, k0 + lane);
      constexpr int J = NB == 1 ? 4 : 2;
      for (int k = k0; k < min(k0 + 32, most_n); k += J) {
        float4 v[kMine][J];
#pragma unroll
        for (int x = 0; x < kMine; ++x)
#pragma unroll
          for (int j = 0; j < J; ++j)
            v[x][j] = k + j < n[x] ? *reinterpret_cast<const float4*>(a.parts + (slot[x] + (int64_t)(k + j) * a.stride) * DIM + at4)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kMine; ++x)
#pragma unroll
          for (int j = 0; j < J; ++j) add(x, __shfl_sync(0xffffffffu, lse[x], (k + j) & 31), v[x][j]);
      }
    }
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      const int i = i1 + x * kWarps;
      if (i >= rows_in) break;
      const float inv = l[x] == 0.f ? 0.f : 1.f / l[x];
      const int64_t at = (r * p.tokens + (i0 + i) / p.group) * (p.heads * p.group) + h * p.group + (i0 + i) % p.group;
      if (lane < DIM / 4)
        *reinterpret_cast<uint2*>(p.o + at * DIM + at4) =
            make_uint2(pack_bf16(o[x].x * inv, o[x].y * inv), pack_bf16(o[x].z * inv, o[x].w * inv));
      if (p.lse && lane == 0) p.lse[at] = l[x] == 0.f ? -INFINITY : (top[x] + log2f(l[x])) * 0.6931471805599453f;
    }
  }
}

// Sizes that both launches go by.
SharedArgs sized(const Kv8Params& p, int beams) {
  SharedArgs a = {};
  a.p = p;
  a.beams = beams;
  const int64_t rows = (int64_t)beams * p.tokens * p.group;
  // As few columns as the rows need: 16 query rows behind 65536 tokens 28 us, in blocks of 32 columns 33;
  // 32 behind 131072 62 us, in blocks of 64 76.  More rows go in blocks of 64, since tiles are
  // loaded and turned into fp16 for each (256 rows behind 16384 tokens 90 us, in blocks of 32 106).  For short
  // lines two blocks of 32 would be faster (45 rows behind 1000 .. 5000 25.5 us, in one of 64 28), but blocks are
  // cut at different keys: a row's roundings would depend on its place in a group of more than 32, not
  // of more than 64, and beams change places.
  a.cw = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  a.blocks = (int)((rows + a.cw - 1) / a.cw);
  a.stride = (int)(rows < a.cw ? rows : a.cw);
  const int64_t tiles = ((int64_t)p.cols * p.page + kKeys - 1) / kKeys * (p.rows / beams) * p.heads * a.blocks;
  a.grid = (int)(tiles < 152 ? tiles : 152);
  return a;
}
// Parts: one for each (group, head, block), and one more for each CTA.
int64_t slots_of(const SharedArgs& a) { return a.p.rows / a.beams * a.p.heads * a.blocks + a.grid; }

template <int MODE, int DIM, int CW>
gdn_status run_common(const SharedArgs& a, cudaStream_t st) {
  auto kern = kv8_common_kernel<MODE, DIM, CW>;
  constexpr int bytes = Room<MODE, DIM, CW>::bytes;
  // once for a device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return GDN_ERR_CUDA;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  kern<<<a.grid, Plan<MODE, CW>::threads, bytes, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int MODE, int DIM>
gdn_status run(SharedArgs& a, cudaStream_t st) {
  const Kv8Params& p = a.p;
  const int64_t rows = (int64_t)p.tokens * p.group;
  // Eight query rows to a CTA where there are no more, or where all CTAs have an SM of their own (15 rows of
  // 30 (row, head) 26.7 us, in one CTA of sixteen 28.2; 16 of 16 16.2 and 18.5), else sixteen, for
  // which a row's own tokens are read once (16 rows of 512 (row, head) with 1000 tokens 95 us, by eights 104; 16 of
  // 128 49.3 and 50.5).
  const int64_t eights = (rows + 7) / 8;
  const bool few = rows <= 8 || p.rows * p.heads * eights <= 152;
  const int64_t y = few ? eights : (rows + 15) / 16;
  if (y > 65535) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (p.pages > 0 && !make_map_3d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, DIM, p.page,
                                  (uint64_t)(2 * p.pages * p.heads), DIM, DIM, p.page,
                                  DIM == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return GDN_ERR_CUDA;
  if (a.grid > 0) {
    const gdn_status s = a.cw == 16   ? run_common<MODE, DIM, 16>(a, st)
                         : a.cw == 32 ? run_common<MODE, DIM, 32>(a, st)
                                      : run_common<MODE, DIM, 64>(a, st);
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
  const cudaError_t e = few ? cudaLaunchKernelEx(&cfg, kv8_own_kernel<MODE, DIM, 1>, a)
                            : cudaLaunchKernelEx(&cfg, kv8_own_kernel<MODE, DIM, 2>, a);
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
