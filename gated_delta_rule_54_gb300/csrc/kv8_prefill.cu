// Attention of many query rows over the 8-bit paged cache, on the tensor cores.
//
// The query rows of a (row, K/V head) are its queries times the query heads that
// share the head, query-major; a CTA takes 256 of them, as two tiles of 128, so
// that one conversion of a block of keys serves both.  Per 128 keys and tile:
//     S = Q K^T   (tcgen05, fp16 x fp16 or 8-bit x E4M3 -> fp32 in TMEM)
//     P = 2^(s - reference)  (two threads per query row; written over S as fp16)
//     O += P V    (tcgen05 with P from TMEM)
// One warp brings the codes of 128 keys by TMA (a box per page); four turn them into
// fp16 (exact), as swizzled operand tiles; one lane of a warp issues the
// products; and eight warps per tile are its rows, two threads to a row.
// E4M3 codes of K are an operand as they arrive; q is then the sum of an E4M3 and an
// E5M2 number, exact for elements down to 2^-13 of the row's largest and off by at most
// 2^-21 of that below (kv8.cuh).  K is not converted, which took the
// second case below from 221 us to 197; the first takes 265 with E4M3 codes.
//
// Measured on a GB300: 4 x 4096 tokens, causal, 16 heads of 128, INT8: 285 us, 0.97
// PFLOP/s; three uneven prompts of up to 2048 tokens against up to 8200 keys, 16 on 4
// heads, E4M3: 197 us, 1.12 PFLOP/s.  Two things bound it.  While a CTA has work the tensor
// pipe is active 46 and 61 % of the time; instruction issue, 2.2 a clock of the four
// schedulers, holds it there with the chain from S by its maxima to P of each tile of rows.
// And the CTAs do not end together: their active cycles are 91 and 77 % of the longest
// one's on average (see Item).  In the
// steps' order (fp16 products), one thread per row (8 warps) took 345 and 258 us, two
// 331 and 240, a CTA per SM for all its items 328 and 249, and one issuing warp for
// both tiles with a shorter conversion 290 and 221.
// Without the exponentials it is 3 to 4 % faster, and with some of them moved to the
// FMA pipe slower.
//
// Scales.  s_j = q . code_j * (scale * ks(block of j)), and V's scale joins the
// exponent: P_j = 2^(s_j + log2 vs - mv), so that fp16 holds it for any scales;
// the denominator takes a block's sum times 2^(mv - log2 vs - m).  That exponent is held
// to 40: a block below it (a V scale that small, or 0) has P below 2^-40, which is 0 in
// fp16, while its sum and the factor stay numbers.  mv follows the
// maximum of s_j + log2 vs only when that grows by more than 2^8 (fp16 has the
// room), and then O is rescaled in TMEM.
#include <cuda.h>

#include "kv8.cuh"
#include "launch.h"
#include "tc.cuh"

namespace gdn {

namespace {

__device__ int g_kv8_prefill_error;

constexpr int kKeys = 128, kRows = 256;
constexpr int kSoftWarps = 16, kConvWarps = 4;
constexpr int kIssuer = kSoftWarps + kConvWarps;  // warp 20 issues, warp 21 loads
constexpr int kThreads = 768;
// registers per thread of the warpgroups: together what the launch gave (6 x 80)
constexpr int kSoftRegs = 96, kConvRegs = 48, kIssueRegs = 48;
static_assert(4 * kSoftRegs + kConvRegs + kIssueRegs == 6 * 80, "register shares");

struct PrefillArgs {
  Kv8Params p;
  CUtensorMap map;  // codes, a page of a head per box
  float* ws;   // splits > 1: parts [block][split][256][DIM + 1 ...]
  int blocks;      // 256-row blocks of a row's queries
  int splits;      // items that share the keys of a block
  unsigned items;  // rows * heads * blocks * splits
};

// fp16 x fp16 -> fp32
constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t lead;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(lead));
  return lead != 0;
}
// Products with descriptors given as the low word (start address and LBO) and the
// common high word, so that stepping through a tile is one 32-bit add.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;  // SBO 1024, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return (saddr >> 4) | (lbo >> 4) << 16;
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
      " setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(kDescHi), "r"((uint32_t)acc));
}
// the same with 8-bit operands, 32 bytes (elements) of a row per product.  In the
// instruction descriptor E4M3 is format 0, as fp16 is there, and E5M2 format 1 (A's: bit 7).
// Rows of 64 bytes: SBO 512, 64-byte swizzle.
constexpr uint32_t kAE5M2 = 1u << 7;
template <int DIM>
__device__ __forceinline__ void umma_ss_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
      " setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(DIM == 128 ? kDescHi : (512u >> 4) | 1u << 14 | 4u << 29), "r"((uint32_t)acc));
}
// A in TMEM: row i in lane i, two fp16 per column
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %4};\n setp.ne.b32 p, %5, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(kDescHi), "r"((uint32_t)acc));
}
// 32 consecutive fp32 columns of this thread's lane; valid after tmem_wait_ld of them
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
        "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// waits for this thread's loads; the values pass through so that no use moves before it
__device__ __forceinline__ void tmem_wait_ld(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                 "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                 "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]),
                 "+f"(v[31])
               :
               : "memory");
}
// two fp32 operations at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15};\n" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// Tile layout: panels of 64 columns, 128-byte rows, 16-byte units swizzled by
// row & 7 (see tc.cuh).  Columns are stored in the order in which kv8_half2 gives
// them: of each four, 0 2 1 3.  Unit u (16 bytes = 8 columns) of a row:
__device__ __forceinline__ uint32_t unit_at(int row, int u) {
  return (uint32_t)((u >> 3) * (kKeys * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4));
}

// 32 bytes, a whole sector at once where the address allows
__device__ __forceinline__ void store32(__nv_bfloat16* to, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// 16 bytes, or zeros; a predicate rather than a branch, so that several of these are
// in flight together
__device__ __forceinline__ uint4 load_if(const __nv_bfloat16* from, bool there) {
  uint4 u;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n"
      " mov.b32 %3, 0;\n @p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(u.x), "=&r"(u.y), "=&r"(u.z), "=&r"(u.w)
      : "l"(from), "r"((int)there));
  return u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One piece of work: up to 256 query rows of a (row, K/V head), and the tiles of
// keys that they see (of which a split has its share).  Later blocks of rows, which see
// more keys, come first, and a CTA takes every gridDim.x-th item.  That does not even the
// CTAs out: it knows neither a row's context nor its tokens.  In units of 128 rows x 128
// keys the file's first case gives a CTA 229 on average (196 to 260, of 6 or 7 items), the
// second 176 (68 to 238, of 1 or 2).
struct Item {
  Kv8Span sp;
  int r, h, row0, here;  // here == 0: nothing
  int ka, nt;
  bool two;
};
__device__ __forceinline__ Item item_of(const PrefillArgs& a, unsigned at) {
  const Kv8Params& p = a.p;
  const unsigned rh = (unsigned)(p.rows * p.heads);
  const int split = at % a.splits;
  const unsigned x = at / a.splits;
  Item m;
  m.row0 = (a.blocks - 1 - (int)(x / rh)) * kRows;
  m.r = (int)(x % rh / (unsigned)p.heads), m.h = (int)(x % rh % (unsigned)p.heads);
  m.sp = kv8_span(p, m.r);
  m.here = max(min(m.sp.n * p.group - m.row0, kRows), 0);
  m.two = m.here > 128;
  m.ka = m.nt = 0;
  if (m.here > 0) {
    int b0, e0, b1, e1;
    kv8_seen(p, m.sp, m.row0 / p.group, b0, e0);
    kv8_seen(p, m.sp, (m.row0 + m.here - 1) / p.group, b1, e1);
    // begins and ends both grow along the rows
    const int ka = b0 / kKeys;
    const int64_t n = e1 > b0 ? (e1 + kKeys - 1) / kKeys - ka : 0;
    m.ka = ka + (int)(n * split / a.splits);
    m.nt = ka + (int)(n * (split + 1) / a.splits) - m.ka;
  }
  return m;
}

// CH: blocks of a tile of keys that have scales of their own (two at least).
// The CTA stays for all its items: the loader and the converters run ahead into the
// next one while the rows of this one finish.
template <int MODE, int DIM, int CH>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(const __grid_constant__ PrefillArgs a) {
  constexpr int kTileBytes = kKeys * DIM * 2;
  constexpr bool F8 = MODE == GDN_QDQ_E4M3;  // scores from the codes as they are
  constexpr uint32_t kCols = 512;  // S0 S1 O0 O1
  constexpr int BK = kKeys / CH;   // keys of a block
  constexpr uint32_t kIdQK = idesc_f16(128, kKeys, 0, 0), kIdPV = idesc_f16(128, DIM, 0, 1);
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t kfull[2], kfree[2], vfull[2], vfree[2];  // by buffer
  __shared__ __align__(8) uint64_t cfull[2][2];                             // codes of K, of V; by buffer
  __shared__ __align__(8) uint64_t qready[2], sfull[2], pready[2], odone[2];  // by tile of rows
  __shared__ float2 meta[4][CH];  // per block of a tile: K scale, log2 of V scale
  __shared__ int valid[4];        // bit c: the block has a page
  __shared__ float row_factor[kRows];
  __shared__ float2 other[2][2][kRows];  // [parity of the tile][half of the keys][row]: maxima
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const Kv8Params& p = a.p;
  const int tid = threadIdx.x, lane = tid % 32;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);  // uniform
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char *sQ = smem, *sK = smem + 2 * kTileBytes;  // sK: K 0, K 1, V 0, V 1
  // Codes arrive where their fp16 tile will be: 128 codes of a row on its second
  // panel, so that a row is read and written over by the same eight lanes.  (Rows
  // of 64 codes have a place of their own.)
  auto codes_at = [&](int kv, int b) {
    return DIM == 128 ? sK + (2 * kv + b) * kTileBytes + kKeys * 128 : smem + 6 * kTileBytes + (2 * kv + b) * kKeys * DIM;
  };

  if (warp == 0) tmem_alloc(&tmem_slot, kCols);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], kConvWarps * 32), mbar_init(&vfull[i], kConvWarps * 32);
      mbar_init(&kfree[i], 1), mbar_init(&vfree[i], 1);
      mbar_init(&cfull[i][0], 1), mbar_init(&cfull[i][1], 1);
      mbar_init(&qready[i], 256), mbar_init(&sfull[i], 1), mbar_init(&pready[i], 256);
      mbar_init(&odone[i], 1);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
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

  if (warp < kSoftWarps) {
    set_regs_up<kSoftRegs>();
    // ======================= rows =======================
    // Two threads per query row, each with half of a tile's keys; they agree on the
    // row's maxima through shared memory.
    const int t = warp / 8, half = (warp / 4) & 1, row = (warp & 3) * 32 + lane, i_row = t * 128 + row;
    constexpr int HK = kKeys / 2, HC = CH / 2;  // a thread's keys, and blocks of them
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 256;\n" ::"r"(1 + t) : "memory"); };
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + t * kKeys, o_col = lane_base + 256 + t * 128 + half * (DIM / 2);
    const bool wide = ((uintptr_t)p.o & 31) == 0;
    // Queries: a warp brings 16 rows of its tile, 16 (or 8) lanes to a row.
    constexpr int kLanes = DIM / 8, kAt = 32 / kLanes;  // lanes of a row, rows at a time
    uint4 q[16 / kAt];
    auto load_q = [&](const Item& m) {
      const int i0 = t * 128 + (warp & 7) * 16 + lane / kLanes;
      int qi = (m.row0 + i0) / p.group, hg = (m.row0 + i0) % p.group;
#pragma unroll
      for (int k = 0; k < 16 / kAt; ++k) {
        q[k] = load_if(p.x + kv8_at(p, m.r, m.sp.base, qi, p.x_row, p.x_token) +
                           (int64_t)(m.h * p.group + hg) * p.x_head + 8 * (lane % kLanes),
                       i0 + k * kAt < m.here);
        for (hg += kAt; hg >= p.group; hg -= p.group) ++qi;
      }
    };
    auto store_q = [&]() {
#pragma unroll
      for (int k = 0; k < 16 / kAt; ++k) {
        const int i = (warp & 7) * 16 + k * kAt + lane / kLanes, u = lane % kLanes;
        float f[8], most = 0.f;
        bf16x8(q[k], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(f[e]));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        float up, back;
        kv8_q_factor<F8 ? 7 : 8>(most, up, back);
        if (u == 0) row_factor[t * 128 + i] = back * fabsf(p.scale) * kLog2eF;
        if (p.scale < 0.f) up = -up;
        if constexpr (F8) {
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float rest[4];
            hi[e] = kv8_q_first(f + 4 * e, up, rest);
            lo[e] = kv8_e5m2x4(rest);
          }
          unsigned char* to = sQ + t * kTileBytes + (u & 1) * 8 +
                              (DIM == 128 ? unit_at(i, u >> 1) : i * 64 + (((u >> 1) ^ (i >> 1 & 3)) << 4));
          *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to + kKeys * DIM) = make_uint2(lo[0], lo[1]);
        } else *reinterpret_cast<uint4*>(sQ + t * kTileBytes + unit_at(i, u)) =
            make_uint4(pack_f16(f[0] * up, f[2] * up), pack_f16(f[1] * up, f[3] * up),
                       pack_f16(f[4] * up, f[6] * up), pack_f16(f[5] * up, f[7] * up));
      }
      fence_proxy_async();
    };
    bool ok = true;
    // tiles of keys that the tile of rows went through, all of the CTA's, and items with any
    uint32_t n = 0, kv_tiles = 0, outs = 0;
    for (unsigned it = blockIdx.x; it < a.items; it += gridDim.x) {
      const Item m = item_of(a, it);
      const bool run = m.here > 0 && (t == 0 || m.two);  // the tile has rows
      if (run) {
        load_q(m);
        store_q();  // (the products that read the item before have completed)
        pair_sync();
        if (m.nt > 0 && ok) mbar_arrive(&qready[t]);
      }
      float l = 0.f, mx = -INFINITY, mv = -INFINITY;
      const float rowfac = row_factor[i_row];
      const bool mine = i_row < m.here;
      const int qi = (m.row0 + i_row) / p.group;
      int beg = 0, end = 0, in0, in1;  // keys of this row, and those that every row of this tile sees
      if (mine) kv8_seen(p, m.sp, qi, beg, end);
      {
        const int last = m.row0 + max(min(t * 128 + 127, m.here - 1), 0);
        int b0, e0, b1, e1;
        kv8_seen(p, m.sp, (m.row0 + t * 128) / p.group, b0, e0);
        kv8_seen(p, m.sp, last / p.group, b1, e1);
        in0 = b1, in1 = e0;
      }
      __syncwarp();
      for (int i = 0; i < m.nt && run; ++i) {
        const uint32_t tile = n + i;
        ok = ok && __all_sync(0xffffffffu, wait(&sfull[t], tile & 1));
        if (!ok) {  // a wait gave up: only the barriers that others may stand at
          pair_sync();
          continue;
        }
        tc_fence_after();
        const int j0 = (m.ka + i) * kKeys + half * HK;
        const uint32_t slot = (kv_tiles + i) & 3;
        const int have = valid[slot] >> (half * HC);
        float v[2][32];
        tmem_ld32(s_col + half * HK, v[0]);
        tmem_ld32(s_col + half * HK + 32, v[1]);
        tmem_wait_ld(v[0]);
        tmem_wait_ld(v[1]);
        if ((have & ((1 << HC) - 1)) != (1 << HC) - 1 || j0 < in0 || j0 + HK > in1) {
          const int first = beg - j0;
          const unsigned len = (unsigned)max(end - beg, 0);
#pragma unroll
          for (int e = 0; e < HK; ++e)
            if ((unsigned)(e - first) >= len || !(have >> (e / BK) & 1)) v[e / 32][e % 32] = -INFINITY;
        }
        // largest product of each block
        float fac[HC], off[HC];
        float nm = -INFINITY, nv = -INFINITY;
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          float top[2];
#pragma unroll
          for (int q4 = 0; q4 < 2; ++q4) {
            top[q4] = v[(c * BK + q4) / 32][(c * BK + q4) % 32];
#pragma unroll
            for (int e = q4 + 2; e + 2 < BK; e += 4)
              top[q4] = max3(top[q4], v[(c * BK + e) / 32][(c * BK + e) % 32], v[(c * BK + e + 2) / 32][(c * BK + e + 2) % 32]);
          }
          // (the chains took all but the last two)
          top[0] = max3(top[0], v[(c * BK + BK - 2) / 32][(c * BK + BK - 2) % 32], v[(c * BK + BK - 1) / 32][(c * BK + BK - 1) % 32]);
          const float2 sc = meta[slot][half * HC + c];
          const float most = fmaxf(top[0], top[1]);
          fac[c] = rowfac * sc.x;
          fac[c] = fac[c] < 1e-30f ? 1e-30f : fac[c];
          off[c] = sc.y;
          const float x = most * fac[c];
          // (a factor of 0, or of NaN where the row sees nothing of the block, would make
          // -inf of a masked key a NaN)
          if (most == -INFINITY) fac[c] = 1e-30f;
          nm = fmaxf(nm, x);
          nv = fmaxf(nv, x + sc.y);
        }
        // (the other thread has its half of S in registers before it comes here, so P
        // may be written over S after this)
        other[i & 1][half][i_row] = make_float2(nm, nv);
        tc_fence_before();
        pair_sync();
        tc_fence_after();
        const float2 o2 = other[i & 1][half ^ 1][i_row];
        nm = fmaxf(fmaxf(nm, o2.x), mx), nv = fmaxf(nv, o2.y);
        const float um = nm == -INFINITY ? 0.f : nm;
        l *= ex2_approx_f(mx - um);
        mx = nm;
        if (__any_sync(0xffffffffu, nv > mv + 8.f)) {
          const float to = fmaxf(mv, nv), f = ex2_approx_f(mv - (to == -INFINITY ? 0.f : to));
          mv = to;
          if (i > 0) {  // the products into O so far have completed with S
#pragma unroll 1
            for (int c = 0; c < DIM / 32; ++c) {
              float w[16];
              tmem_ld16(o_col + 16 * c, w);
              uint32_t u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(w[e] * f);
              tmem_st16(o_col + 16 * c, u);
            }
          }
        }
        const float uv = mv == -INFINITY ? 0.f : mv;
#pragma unroll
        for (int c = 0; c < HC; ++c) off[c] = fmaxf(off[c] - uv, -um - 40.f);
        float2 sum[HC];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const int b = (32 * c + e) / BK;
            const float2 x = fma2(make_float2(v[c][e], v[c][e + 1]), make_float2(fac[b], fac[b]),
                                  make_float2(off[b], off[b]));
            const float2 w = make_float2(ex2_approx_f(x.x), ex2_approx_f(x.y));
            sum[b] = (32 * c + e) % BK == 0 ? w : add2(sum[b], w);
            pk[e / 2] = pack_f16(w.x, w.y);
          }
          tmem_st16(s_col + half * (HK / 2) + 16 * c, pk);
        }
#pragma unroll
        for (int c = 0; c < HC; ++c) l = fmaf(sum[c].x + sum[c].y, ex2_approx_f(-off[c] - um), l);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&pready[t]);
      }

      if (run) {
        // ---- outputs: each thread half of its row's dims ----
        // the row's sum, in the order of the keys
        pair_sync();
        other[0][half][i_row].x = l;
        pair_sync();
        l = other[0][0][i_row].x + other[0][1][i_row].x;
        const bool any = m.nt > 0;
        if (any) {
          ok = ok && __all_sync(0xffffffffu, wait(&odone[t], outs & 1));
          tc_fence_after();
        }
        // l is 0 where no key is seen, and NaN where a score is
        const float fac = kv8_out_factor<MODE>(mv, mx, l);
        const float lse2 = l == 0.f ? -INFINITY : mx + log2f(l);
        const int64_t at = (m.sp.base + qi) * (p.heads * p.group) + m.h * p.group + (m.row0 + i_row) % p.group;
        float* part = a.ws + ((int64_t)it * kRows + i_row) * (DIM + 4);
        if (ok) {
#pragma unroll
          for (int c = 0; c < DIM / 64; ++c) {
            float v[32];
            if (any) {
              __syncwarp();
              tmem_ld32(o_col + 32 * c, v);
              tmem_wait_ld(v);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = 0.f;
            }
            if (mine) {
              // columns 4 i .. 4 i + 3 are dims 4 i + (0 2 1 3); where nothing was seen the
              // factor is 0 and O holds finite sums or zeros
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                const int d = half * (DIM / 2) + 32 * c + e;
                if (a.splits == 1) {
                  uint32_t w[8];
#pragma unroll
                  for (int f = 0; f < 16; f += 4)
                    w[f / 2] = pack_bf16(v[e + f] * fac, v[e + f + 2] * fac),
                    w[f / 2 + 1] = pack_bf16(v[e + f + 1] * fac, v[e + f + 3] * fac);
                  store32(p.o + at * DIM + d, w, wide);
                } else {
#pragma unroll
                  for (int f = 0; f < 16; f += 4)
                    *reinterpret_cast<float4*>(part + d + f) =
                        make_float4(v[e + f] * fac, v[e + f + 2] * fac, v[e + f + 1] * fac, v[e + f + 3] * fac);
                }
              }
            }
          }
          if (mine && half == 0) {
            if (a.splits > 1) part[DIM] = lse2;
            else if (p.lse) p.lse[at] = lse2 * 0.6931471805599453f;
          }
        }
        tc_fence_before();  // O has been read: the next item's products may write it (after P's signal)
        if (any) ++outs;
        n += m.nt;
      }
      kv_tiles += m.nt;
    }
  } else if (warp < kIssuer) {
    set_regs_down<kConvRegs>();
    // ======================= codes to fp16 =======================
    // a lane takes 16 codes at a time; the two rows of eight neighbouring lanes are
    // chosen so that their loads and their stores each fall on different banks
    const int cw = warp - kSoftWarps;
    constexpr int kPer = DIM / 16, kStep = 2048 / DIM;
    const int unit = DIM == 128 ? (lane & 3) | ((lane >> 3) & 1) << 2 : lane & 3;
    const int r8 = DIM == 128 ? (lane >> 4 & 1) * 2 : lane >> 2;
    // 128-byte rows: (0 5) (1 4) (2 7) (3 6), the even warps the first of each two pairs
    const int row0c = DIM == 128 ? (cw / 2) * 8 + (((r8 + (cw & 1)) ^ ((lane >> 2 & 1) ? 5 : 0)))
                                 : cw * 8 + r8;
    const int from0 = DIM == 128 ? row0c * 128 + ((unit ^ (row0c & 7)) << 4)
                                 : row0c * 64 + ((unit ^ (row0c >> 1 & 3)) << 4);
    const uint32_t to0 = unit_at(row0c, 2 * unit), to1 = unit_at(row0c, 2 * unit + 1);
    uint32_t n = 0;  // tiles so far
    bool ok = true;
    for (unsigned it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const int nt = item_of(a, it).nt;
#pragma unroll 1
      for (int x = F8; x < 2 * nt && ok; x += 1 + F8) {  // K, V, K, V, ...; or V alone
        const int kv = F8 ? 1 : x & 1;
        const uint32_t tile = n + (x >> 1), b = tile & 1;
        ok = wait(&cfull[kv][b], (tile >> 1) & 1);
        if (!ok) break;
        unsigned char* to = sK + (2 * kv + b) * kTileBytes;
        const unsigned char* from = codes_at(kv, b);
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
      n += nt;
    }
  } else {
    set_regs_down<kIssueRegs>();
  }
  if (warp == kIssuer + 1) {
    // ======================= codes by TMA =======================
    const int boxes = kKeys >> p.shift;
    uint32_t n = 0;  // tiles so far
    int issued[2] = {0, 0};
    bool ok = true;
    for (unsigned it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item m = item_of(a, it);
      // (this warp is two tiles of keys ahead of the rows: their queries may come near)
      for (int i = lane; i < m.here && it != blockIdx.x; i += 32) {
        const int qi = (m.row0 + i) / p.group;
        const __nv_bfloat16* x = p.x + kv8_at(p, m.r, m.sp.base, qi, p.x_row, p.x_token) +
                                 (int64_t)(m.h * p.group + (m.row0 + i) - qi * p.group) * p.x_head;
#pragma unroll
        for (int d = 0; d < DIM; d += 64) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(x + d));
      }
      // page ids and scales are asked for a tile before
      auto page_of = [&](int i) {
        const int j = (m.ka + i) * kKeys + (lane << p.shift);
        return lane < boxes && i < m.nt && j < m.sp.end ? p.table[(int64_t)m.r * p.cols + (j >> p.shift)] : -1;
      };
      auto scale_of = [&](int id) {
        if (id < 0 || id >= p.pages) return make_float2(0.f, 0.f);
        const int64_t tile = (int64_t)id * p.heads + m.h;
        return make_float2(p.scales[tile], p.scales[tile + p.pages * p.heads]);
      };
      int id = page_of(0), id1 = page_of(1);
      float2 sc = scale_of(id);
      for (int i = 0; i < m.nt; ++i) {
        const uint32_t tile = n + i, b = tile & 1;
        const bool have = id >= 0 && id < p.pages;
        // block c of the scales lies in page c >> (log2 of blocks per page)
        const int from = (lane * BK) >> p.shift;
        const float ks = __shfl_sync(0xffffffffu, sc.x, from & 31);
        const float vs = __shfl_sync(0xffffffffu, sc.y, from & 31);
        const bool there = __shfl_sync(0xffffffffu, (int)have, from & 31);
        const unsigned bits = __ballot_sync(0xffffffffu, there && lane < CH);
        const unsigned bytes = __popc(__ballot_sync(0xffffffffu, have)) * (DIM << p.shift);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && __all_sync(0xffffffffu, wait(kv ? &vfree[b] : &kfree[b], ((tile >> 1) & 1) ^ 1));
          if (!ok) break;
          if (kv == 0) {
            if (lane < CH) meta[tile & 3][lane] = there ? kv8_scales(ks, vs) : make_float2(0.f, -INFINITY);
            if (lane == 0) valid[tile & 3] = (int)bits;
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(&cfull[kv][b], bytes);
          __syncwarp();
          issued[kv] = (int)tile + 1;
          if (have)
            tma_load_3d(codes_at(kv, b) + (lane << p.shift) * DIM, &a.map, 0, 0,
                        (int)((kv * p.pages + id) * p.heads + m.h), &cfull[kv][b]);
        }
        if (!ok) break;
        id = id1;
        sc = scale_of(id);
        id1 = page_of(i + 2);
      }
      n += m.nt;
    }
    // no copy is in flight when the CTA ends, whatever ended the loop
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      for (int i = max(issued[kv] - 2, 0); i < issued[kv]; ++i) mbar_wait(&cfull[kv][i & 1], (i >> 1) & 1);
  } else if (warp == kIssuer) {
    // ======================= products =======================
    // The tiles of rows in turn: P V of one block of keys, then Q K^T of the next; so
    // one tile's products run while the other's rows compute.  (With a warp for each
    // tile they fall into step, and the tensor cores wait for both.)  The whole warp
    // goes through this, so that descriptors stay in uniform registers; one elected
    // lane issues.
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    const uint32_t dq = desc_lo(base, 16);
    const uint32_t dk = desc_lo(base + (uint32_t)((F8 ? codes_at(0, 0) : sK) - smem), 16);
    constexpr uint32_t kKStep = (F8 && DIM == 64 ? kKeys * DIM : kTileBytes) >> 4;
    uint64_t* kthere = F8 ? &cfull[0][0] : &kfull[0];  // K's operand of a buffer
    const uint32_t dv = desc_lo(base + 4 * kTileBytes, kKeys * 128);
    constexpr uint32_t kTileStep = kTileBytes >> 4;
    const bool lead = elect_one();
    auto qk = [&](int t, uint32_t b) {
      const uint32_t k = dk + b * kKStep, q = dq + t * kTileStep;
      if (lead) {
#pragma unroll
        for (int s = 0; s < DIM / 16; ++s) {
          constexpr int kRow = F8 ? DIM / 32 : 4;  // products along a row of an operand's panel
          const uint32_t at = s % kRow * 32 >> 4, off = (s / kRow * (kKeys * (F8 ? DIM : 128)) >> 4) + at;
          if constexpr (F8)  // q's first parts, then its second ones, with the same codes
            umma_ss_f8<DIM>(tm + t * kKeys, q + off, k + at, kIdQK | (s < kRow ? 0 : kAE5M2), s > 0);
          else
            umma_ss(tm + t * kKeys, q + off, k + off, kIdQK, s > 0);
        }
        umma_commit(&sfull[t]);
      }
      __syncwarp();
    };
    auto pv = [&](int t, uint32_t b, bool add) {
      const uint32_t v = dv + b * kTileStep;
      if (lead) {
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)
          umma_ts(tm + 256 + t * 128, tm + t * kKeys + 8 * s, v + s * (2048 >> 4), kIdPV, add || s > 0);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (lead) umma_commit(bar);
      __syncwarp();
    };
    auto all_wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait(bar, parity));
    };
    uint32_t n = 0, done[2] = {0, 0}, outs[2] = {0, 0};  // tiles of keys; by tile of rows: those, and items
    bool ok = true;
    for (unsigned it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item m = item_of(a, it);
      if (m.nt == 0) continue;
      ok = all_wait(&kthere[n & 1], (n >> 1) & 1) && all_wait(&qready[0], outs[0] & 1);
      tc_fence_after();
      if (ok) qk(0, n & 1);
      if (m.two) {
        ok = ok && all_wait(&qready[1], outs[1] & 1);
        tc_fence_after();
        if (ok) qk(1, n & 1);
      }
      if (ok) commit(&kfree[n & 1]);
      for (int i = 0; i < m.nt && ok; ++i) {
        const uint32_t tile = n + i, b = tile & 1;
        const bool more = i + 1 < m.nt;
        ok = all_wait(&vfull[b], (tile >> 1) & 1);
        if (more) ok = ok && all_wait(&kthere[b ^ 1], ((tile + 1) >> 1) & 1);
        ok = ok && all_wait(&pready[0], (done[0] + i) & 1);
        if (!ok) break;
        tc_fence_after();
        pv(0, b, i > 0);
        if (more) qk(0, b ^ 1);
        if (m.two) {
          ok = all_wait(&pready[1], (done[1] + i) & 1);
          if (!ok) break;
          tc_fence_after();
          pv(1, b, i > 0);
          if (more) qk(1, b ^ 1);
        }
        commit(&vfree[b]);
        if (more) commit(&kfree[b ^ 1]);
      }
      commit(&odone[0]);  // completes with every product issued so far
      done[0] += m.nt, ++outs[0];
      if (m.two) {
        commit(&odone[1]);
        done[1] += m.nt, ++outs[1];
      }
      n += m.nt;
    }
    if (outs[0] > 0) wait(&odone[0], (outs[0] - 1) & 1);
    if (outs[1] > 0) wait(&odone[1], (outs[1] - 1) & 1);
  } else if (warp > kIssuer + 1 && p.cu) {
    constexpr int kIdle = kThreads / 32 - kIssuer - 2;  // warps without another role
    kv8_fill<DIM>(p, (int64_t)blockIdx.x * kIdle + warp - kIssuer - 2, (int64_t)gridDim.x * kIdle, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && abort_flag) atomicOr(&g_kv8_prefill_error, 1);
  if (warp == 0) tmem_dealloc(tmem, kCols);
}

// Joins the parts of a block's rows: one warp per row, in order of the splits.
template <int DIM>
__global__ void __launch_bounds__(256) kv8_prefill_join_kernel(const __grid_constant__ PrefillArgs a) {
  const Kv8Params& p = a.p;
  const int lane = threadIdx.x % 32, i = blockIdx.y * 8 + threadIdx.x / 32;
  const int64_t rh = p.rows * p.heads, x = blockIdx.x;
  const int block = a.blocks - 1 - (int)(x / rh);
  const int64_t r = x % rh / p.heads;
  const int h = (int)(x % rh % p.heads);
  const Kv8Span sp = kv8_span(p, r);
  const int64_t row = (int64_t)block * kRows + i;
  if (row >= (int64_t)sp.n * p.group) return;
  const float* part = a.ws + (x * a.splits * kRows + i) * (DIM + 4);
  constexpr int64_t step = (int64_t)kRows * (DIM + 4);
  float top = -INFINITY;
  for (int s = 0; s < a.splits; ++s) top = max_nan(top, part[s * step + DIM]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int s = 0; s < a.splits && top != -INFINITY; ++s) {
    const float c = ex2_approx_f(part[s * step + DIM] - top);
    l += c;
    if (lane < DIM / 4) {
      const float4 v = *reinterpret_cast<const float4*>(part + s * step + 4 * lane);
      o.x = fmaf(c, v.x, o.x), o.y = fmaf(c, v.y, o.y), o.z = fmaf(c, v.z, o.z), o.w = fmaf(c, v.w, o.w);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (sp.base + row / p.group) * (p.heads * p.group) + h * p.group + row % p.group;
  if (lane < DIM / 4)
    *reinterpret_cast<uint2*>(p.o + at * DIM + 4 * lane) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

int64_t blocks_of(const Kv8Params& p) {
  return ((int64_t)p.tokens * p.group + kRows - 1) / kRows;
}
// CTAs per block of rows: where the blocks do not fill 152 SMs, the keys are
// split, down to two tiles each (in us, split / whole: 256 tokens x 4 heads of one K/V head
// on 8192 keys 26/114; 512 x 4 of four on 4096 31/62; 64 x 4 of two on 700 19/20)
int splits_of(const Kv8Params& p) {
  int64_t keys = (int64_t)p.cols * p.page;
  if (p.window > 0 && (int64_t)p.window + p.tokens < keys) keys = (int64_t)p.window + p.tokens;
  const int64_t ctas = blocks_of(p) * p.rows * p.heads, tiles = (keys + kKeys - 1) / kKeys;
  int64_t n = ctas > 0 ? 152 / ctas : 1;
  if (n > tiles / 2) n = tiles / 2;
  return n < 1 ? 1 : (int)n;
}

template <int MODE, int DIM, int CH>
gdn_status run(PrefillArgs& a, cudaStream_t st) {
  const Kv8Params& p = a.p;
  a.map = CUtensorMap();
  if (p.pages > 0 &&
      !make_map_3d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, DIM, p.page,
                   (uint64_t)(2 * p.pages * p.heads), DIM, DIM, p.page,
                   DIM == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return GDN_ERR_CUDA;
  const int64_t blocks = (int64_t)a.blocks * p.rows * p.heads;
  if (blocks * a.splits > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED_SHAPE;
  constexpr int bytes = 6 * kKeys * DIM * 2 + (DIM == 128 ? 0 : 4 * kKeys * DIM) + 1024;
  auto kern = kv8_prefill_kernel<MODE, DIM, CH>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return GDN_ERR_CUDA;
  a.items = (unsigned)(blocks * a.splits);
  kern<<<a.items < 152 ? a.items : 152, kThreads, bytes, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  if (a.splits == 1) return GDN_OK;
  kv8_prefill_join_kernel<DIM><<<dim3((unsigned)blocks, kRows / 8), 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

size_t kv8_prefill_workspace(const Kv8Params& p, int dim) {
  const int splits = splits_of(p);
  if (splits == 1) return 0;
  return (size_t)(blocks_of(p) * p.rows * p.heads) * splits * kRows * (dim + 4) * sizeof(float);
}

gdn_status launch_kv8_prefill(const Kv8Params& p, int mode, int dim, void* workspace,
                              cudaStream_t st) {
  PrefillArgs a;
  a.p = p;
  a.ws = static_cast<float*>(workspace);
  a.blocks = (int)blocks_of(p);
  a.splits = splits_of(p);
  // pages of 64 and 128 tokens: two scales per tile of keys instead of eight (4 x 4096
  // tokens, pages of 64: 280 us, with eight 295)
  auto pick = [&](auto two, auto eight) { return p.page >= 64 ? two(a, st) : eight(a, st); };
  if (mode == GDN_QDQ_E4M3)
    return dim == 128 ? pick(run<GDN_QDQ_E4M3, 128, 2>, run<GDN_QDQ_E4M3, 128, 8>)
                      : pick(run<GDN_QDQ_E4M3, 64, 2>, run<GDN_QDQ_E4M3, 64, 8>);
  return dim == 128 ? pick(run<GDN_QDQ_INT8, 128, 2>, run<GDN_QDQ_INT8, 128, 8>)
                    : pick(run<GDN_QDQ_INT8, 64, 2>, run<GDN_QDQ_INT8, 64, 8>);
}

int kv8_prefill_device_error(bool reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv8_prefill_error, sizeof(int)) != cudaSuccess) return -1;
  if (reset && v) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_kv8_prefill_error, &z, sizeof(int)) != cudaSuccess) return -1;
  }
  return v;
}

}  // namespace gdn
