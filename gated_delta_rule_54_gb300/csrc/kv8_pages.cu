// Pages of the 8-bit cache: fork, reserve, compact and copy.
//
// Each of fork, reserve and compact is one plan and one mover.  The plan works
// on the small arrays only (reference counts, tables, lengths): one cluster of
// CTAs, whose phases are separated by cluster barriers, so that choosing the
// n lowest free pages (a scan of all counts) and rewriting the tables need no
// further launches and no word from the host.  The mover copies whole pages in
// all planes from the list that the plan left in the workspace; it is bound by
// HBM (each byte read once and written once).
//
// Measured on a GB300, 128 rows, 8000 pages, 4 layers of 4 heads: plan 12 us, mover 7
// us; compacting 500 pages 9 and 5 us.  Latency bounds both: the plan is a chain of
// cluster barriers and trips to L2 (the rows' small arrays in shared memory took
// 15 us to 12), and there are few pages to move.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace gdn {

namespace {

constexpr int kCtas = 8, kPlanThreads = 1024, kPlanWarps = kCtas * kPlanThreads / 32;
constexpr int kMaxRows = 4096;

enum Op { kFork = 0, kReserve = 1, kCompact = 2 };

struct PlanParams {
  const int32_t *table, *lengths, *refs, *parents, *extra;
  const uint8_t* drop;
  int32_t *table_out, *lengths_out, *refs_out, *count_out;  // count_out: missing or live
  // workspace: number of moves, their sources and destinations; free pages in
  // order (fork, reserve) or each page's rank among the moved (compact)
  int32_t *n_moves, *src, *dst, *list;
  int64_t pages, rows;
  int cols, page;
};

__device__ __forceinline__ int pages_of(int len, int page) {
  return len <= 0 ? 0 : (int)(((int64_t)len + page - 1) / page);
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Exclusive prefix over all warps of the cluster of one count per warp; total
// in `all`.  cnt: this CTA's [32] shared counts.
__device__ __forceinline__ int warp_prefix(cg::cluster_group& cl, int (*cnt), int value, int& all) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) cnt[warp] = value;
  cl.sync();
  int before = 0, sum = 0;
  const int me = (int)cl.block_rank() * 32 + warp;
  for (int c = 0; c < kCtas; ++c) {
    const int x = cl.map_shared_rank(cnt, c)[lane];
    before += c * 32 + lane < me ? x : 0;
    sum += x;
  }
  all = warp_sum(sum);
  before = warp_sum(before);
  cl.sync();  // the counts may be written again
  return before;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kPlanThreads)
    kv8_compact_kernel(const PlanParams p) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int cnt[32];
  const int tid = threadIdx.x, lane = tid % 32;
  const int gtid = (int)cl.block_rank() * kPlanThreads + tid, gwarp = gtid / 32;
  const int rows = (int)p.rows;
  const int64_t P = p.pages;
  // this warp's pages of a scan: a contiguous range, a multiple of 32 long
  const int64_t span = ((P + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
  const int64_t p0 = gwarp * span < P ? gwarp * span : P, p1 = p0 + span < P ? p0 + span : P;

  int live = 0;
  for (int64_t i = p0 + lane; i < p1; i += 32) live += p.refs[i] > 0;
  int n;
  const int before = warp_prefix(cl, cnt, warp_sum(live), n);
  // live pages below n: the warp whose range holds page n knows
  int below = 0;
  if (p0 <= n && n < p1) {
    for (int64_t i = p0 + lane; i < n; i += 32) below += p.refs[i] > 0;
    below = before + warp_sum(below);
  }
  int low;
  warp_prefix(cl, cnt, below, low);
  const int moved = n >= P ? 0 : n - low;  // = free pages below n = live pages from n on
  // rank of every free page below n and of every live page from n on
  int seen = before;
  for (int64_t i = p0; i < p1; i += 32) {
    const bool alive = i + lane < p1 && p.refs[i + lane] > 0;
    const unsigned mask = __ballot_sync(0xffffffffu, alive);
    const int64_t pg = i + lane;
    const int lb = seen + __popc(mask & ((1u << lane) - 1));  // live pages before pg
    if (pg < p1 && n < P) {
      if (pg < n && !alive) p.dst[(int)(pg - lb)] = (int)pg;
      if (pg >= n && alive) {
        const int rank = moved - n + lb;
        p.src[rank] = (int)pg;
        p.list[pg] = rank;
      }
    }
    seen += __popc(mask);
  }
  cl.sync();
  if (gtid == 0) *p.n_moves = moved, *p.count_out = n;
  // counts move with the pages
  for (int64_t i = gtid; i < P; i += kCtas * kPlanThreads)
    if (i >= n) p.refs_out[i] = 0;
    else if (p.refs[i] > 0) p.refs_out[i] = p.refs[i];
  for (int i = gtid; i < moved; i += kCtas * kPlanThreads) p.refs_out[p.dst[i]] = p.refs[p.src[i]];
  for (int r = gwarp; r < rows; r += kPlanWarps) {
    const int own = pages_of(p.lengths[r], p.page);
    for (int c = lane; c < p.cols; c += 32) {
      int pg = c < own ? p.table[(int64_t)r * p.cols + c] : -1;
      if (pg < 0 || pg >= P) pg = -1;
      else if (pg >= n) pg = p.refs[pg] > 0 ? p.dst[p.list[pg]] : -1;
      p.table_out[(int64_t)r * p.cols + c] = pg;
    }
  }
}

template <int OP>
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kPlanThreads)
    kv8_plan_kernel(const PlanParams p) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int cnt[32];
  // small arrays of all rows, in every CTA.  s_a: fork's children of a row, then the
  // pages wanted by the rows before a row; s_b: fork's first child of a row; and the
  // lengths, the parents (fork) or the extra tokens (reserve).
  extern __shared__ int s_rows[];
  int *s_a = s_rows, *s_b = s_a + p.rows, *s_len = s_b + p.rows, *s_par = s_len + p.rows;
  __shared__ int64_t s_total, s_over;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int gtid = (int)cl.block_rank() * kPlanThreads + tid, gwarp = gtid / 32;
  const int rows = (int)p.rows;
  const int64_t P = p.pages;
  // this warp's pages of a scan: a contiguous range, a multiple of 32 long
  const int64_t span = ((P + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
  const int64_t p0 = gwarp * span < P ? gwarp * span : P, p1 = p0 + span < P ? p0 + span : P;

  // ---- fork, reserve: reference counts of what stays --------------------
  for (int64_t i = gtid; i < P; i += kCtas * kPlanThreads) p.refs_out[i] = p.refs[i];
  for (int r = tid; r < rows; r += kPlanThreads) {
    s_len[r] = max(p.lengths[r], 0);
    if constexpr (OP == kFork) {
      const int q = p.drop ? (p.drop[r] ? -1 : r) : p.parents[r];
      s_par[r] = q >= 0 && q < rows ? q : -1;
      s_a[r] = 0, s_b[r] = rows;
    } else {
      s_par[r] = max(p.extra[r], 0);
    }
  }
  __syncthreads();
  if constexpr (OP == kFork) {
    for (int r = tid; r < rows; r += kPlanThreads) {
      const int q = s_par[r];
      if (q >= 0) atomicAdd(&s_a[q], 1), atomicMin(&s_b[q], r);
    }
    cl.sync();  // counts copied, children known
    for (int r = gwarp; r < rows; r += kPlanWarps) {
      const int len = s_len[r], own = min(pages_of(len, p.page), p.cols), kids = s_a[r];
      for (int c = lane; c < own; c += 32) {
        const bool whole = (int64_t)(c + 1) * p.page <= len;
        const int more = (whole ? kids : min(kids, 1)) - 1;
        const int pg = p.table[(int64_t)r * p.cols + c];
        if (more != 0 && pg >= 0 && pg < P) atomicAdd(&p.refs_out[pg], more);
      }
    }
  }
  // reserve: pages of a row's longer sequence
  auto need = [&](int r) {
    return (int)(((int64_t)s_len[r] + s_par[r] + p.page - 1) / p.page);
  };
  // fresh pages wanted by a row
  auto wanted = [&](int r) {
    if constexpr (OP == kFork) {
      const int q = s_par[r];
      return q >= 0 && s_len[q] % p.page != 0 && s_b[q] != r && pages_of(s_len[q], p.page) <= p.cols ? 1 : 0;
    } else {
      return min(need(r), p.cols) - min(pages_of(s_len[r], p.page), p.cols);
    }
  };
  // a scan by one warp of each CTA, in 64 bits: 4096 rows may want up to 2^27 pages each.  A
  // row's place in it stops at 2^30, as many as a pool can have
  __syncthreads();  // the children have been read
  if (warp == 0) {
    int64_t run = 0, over = 0;
    for (int r0 = 0; r0 < rows; r0 += 32) {
      const int r = r0 + lane;
      const int64_t w = r < rows ? wanted(r) : 0;
      int64_t x = w;
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (r < rows) s_a[r] = (int)min(run + x - w, (int64_t)1 << 30);
      run += __shfl_sync(0xffffffffu, x, 31);
      if constexpr (OP == kReserve)
        if (r < rows) over += max(need(r) - max(p.cols, pages_of(s_len[r], p.page)), 0);
    }
    if constexpr (OP == kReserve)
      for (int d = 16; d; d >>= 1) over += __shfl_xor_sync(0xffffffffu, over, d);
    if (lane == 0) s_total = run, s_over = over;
  }
  cl.sync();  // counts settled, wanted pages known
  const int64_t total = s_total;
  // ---- the lowest free pages --------------------------------------------
  int free_ = 0;
  if (total > 0)
    for (int64_t i = p0 + lane; i < p1; i += 32) free_ += p.refs_out[i] == 0;
  int all;
  int rank = warp_prefix(cl, cnt, warp_sum(free_), all);
  if (total > 0)
    for (int64_t i = p0; i < p1 && rank < total; i += 32) {
      const bool f = i + lane < p1 && p.refs_out[i + lane] == 0;
      const unsigned mask = __ballot_sync(0xffffffffu, f);
      const int k = rank + __popc(mask & ((1u << lane) - 1));
      if (f && k < total) p.list[k] = (int)(i + lane);
      rank += __popc(mask);
    }
  cl.sync();
  const int have = all < total ? all : (int)total;
  for (int i = gtid; i < have; i += kCtas * kPlanThreads) p.refs_out[p.list[i]] = 1;
  if (gtid == 0) *p.count_out = (int)min(total - have + s_over, (int64_t)0x7fffffff), *p.n_moves = OP == kFork ? have : 0;
  for (int r = gwarp; r < rows; r += kPlanWarps) {
    if constexpr (OP == kFork) {
      const int q = s_par[r], len = q >= 0 ? s_len[q] : 0;
      const int own = min(pages_of(len, p.page), p.cols), k = s_a[r];
      const bool fresh = wanted(r) > 0;
      for (int c = lane; c < p.cols; c += 32) {
        int pg = c < own ? p.table[(int64_t)q * p.cols + c] : -1;
        if (fresh && c == own - 1) {
          if (k < have) {
            const int to = p.list[k];
            // a page id that is not one has nothing to copy: the row's page stays empty
            p.src[k] = pg >= 0 && pg < P ? pg : to;
            p.dst[k] = to;
            pg = to;
          } else {
            pg = -1;
          }
        }
        p.table_out[(int64_t)r * p.cols + c] = pg;
      }
      if (lane == 0) p.lengths_out[r] = len;
    } else {
      const int64_t len = s_len[r], ex = s_par[r];
      const int own = min(pages_of((int)len, p.page), p.cols), k = s_a[r], w = wanted(r);
      for (int c = lane; c < p.cols; c += 32) {
        int pg = c < own ? p.table[(int64_t)r * p.cols + c] : -1;
        if (c >= own && c < own + w) pg = k + c - own < have ? p.list[k + c - own] : -1;
        p.table_out[(int64_t)r * p.cols + c] = pg;
      }
      // no row grows past its table (one that was longer already stays so)
      if (lane == 0) p.lengths_out[r] = (int)max(len, min(len + ex, (int64_t)p.cols * p.page));
    }
  }
}

// Copies pages src[i] -> dst[i], i < n (or *n_dev), in all planes: 16 KiB of a
// page per CTA step, then the scales of a (page, plane).
struct MoveParams {
  uint8_t* codes;
  float* scales;
  const int32_t *src, *dst, *n_dev;
  int64_t pages, n, bytes;  // bytes of a page in one plane
  int planes, heads, parts;
};

constexpr int kMoveThreads = 256, kMoveBytes = kMoveThreads * 16 * 4;

__global__ void __launch_bounds__(kMoveThreads) kv8_move_kernel(const MoveParams p) {
  grid_dep_wait();
  const int64_t n = p.n_dev ? *p.n_dev : p.n;
  const int64_t items = n * p.planes * p.parts;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int part = (int)(it % p.parts);
    const int64_t pl = it / p.parts % p.planes, i = it / p.parts / p.planes;
    const int64_t s = p.src[i], d = p.dst[i];
    if (s == d || s < 0 || d < 0 || s >= p.pages || d >= p.pages) continue;
    const int64_t off = (int64_t)part * kMoveBytes;
    const uint8_t* a = p.codes + (pl * p.pages + s) * p.bytes + off;
    uint8_t* b = p.codes + (pl * p.pages + d) * p.bytes + off;
    const int64_t left = p.bytes - off;
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = ((int64_t)j * kMoveThreads + threadIdx.x) * 16;
      if (at < left) u[j] = *reinterpret_cast<const uint4*>(a + at);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = ((int64_t)j * kMoveThreads + threadIdx.x) * 16;
      if (at < left) *reinterpret_cast<uint4*>(b + at) = u[j];
    }
    if (part == 0)
      for (int h = threadIdx.x; h < p.heads; h += kMoveThreads)
        p.scales[(pl * p.pages + d) * p.heads + h] = p.scales[(pl * p.pages + s) * p.heads + h];
  }
}

gdn_status validate_pool(const gdn_kv8_pool* p) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->pages < 0 || p->rows <= 0 || p->cols < 0 || p->planes <= 0 || p->heads <= 0)
    return GDN_ERR_INVALID_ARG;
  if (p->page != 16 && p->page != 32 && p->page != 64 && p->page != 128)
    return GDN_ERR_UNSUPPORTED_SHAPE;
  if (p->dim != 64 && p->dim != 128) return GDN_ERR_UNSUPPORTED_SHAPE;
  if (p->rows > kMaxRows || (int64_t)p->cols * p->page > 0x7fffffffLL || p->pages > (1LL << 30))
    return GDN_ERR_UNSUPPORTED_SHAPE;
  return GDN_OK;
}

gdn_status launch_move(const gdn_kv8_pool& p, uint8_t* codes, float* scales, const int32_t* src,
                       const int32_t* dst, const int32_t* n_dev, int64_t n, int64_t most,
                       bool after_plan, cudaStream_t st) {
  MoveParams m;
  m.codes = codes, m.scales = scales, m.src = src, m.dst = dst, m.n_dev = n_dev, m.n = n;
  m.pages = p.pages, m.planes = p.planes, m.heads = p.heads;
  m.bytes = (int64_t)p.heads * p.page * p.dim;
  m.parts = (int)((m.bytes + kMoveBytes - 1) / kMoveBytes);
  const int64_t items = most * m.planes * m.parts;
  if (items == 0) return GDN_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < 152 * 8 ? items : 152 * 8));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_plan ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv8_move_kernel, m) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// Workspace: [0] moves; then src, dst, list.  Fork moves at most one page per
// row and lists as many; reserve lists at most rows * cols; compact moves at
// most half the pages and ranks them all.
size_t list_ints(const gdn_kv8_pool& p) {
  const size_t rc = (size_t)p.rows * (p.cols > 0 ? p.cols : 1);
  return rc > (size_t)p.pages ? rc : (size_t)p.pages;
}
size_t move_ints(const gdn_kv8_pool& p) {
  return (size_t)(p.rows > p.pages ? p.rows : p.pages);
}

gdn_status run_plan(int op, const gdn_kv8_pool& pool, PlanParams p, void* workspace,
                    cudaStream_t st) {
  int32_t* w = static_cast<int32_t*>(workspace);
  p.n_moves = w;
  p.src = w + 4;
  p.dst = p.src + move_ints(pool);
  p.list = p.dst + move_ints(pool);
  p.pages = pool.pages, p.rows = pool.rows, p.cols = pool.cols, p.page = pool.page;
  if (op == kCompact) {
    kv8_compact_kernel<<<kCtas, kPlanThreads, 0, st>>>(p);
  } else {
    auto kern = op == kFork ? kv8_plan_kernel<kFork> : kv8_plan_kernel<kReserve>;
    const int bytes = 16 * (int)pool.rows;  // at most 64 KiB
    if (bytes > 47 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return GDN_ERR_CUDA;
    kern<<<kCtas, kPlanThreads, bytes, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

bool misaligned(std::initializer_list<const void*> ptrs, uintptr_t mask) {
  for (const void* q : ptrs)
    if ((uintptr_t)q & mask) return true;
  return false;
}

}  // namespace

}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_kv8_pool_workspace_bytes(const gdn_kv8_pool* p) {
  if (validate_pool(p) != GDN_OK) return 0;
  return 4 * (4 + 2 * move_ints(*p) + list_ints(*p));
}

gdn_status gdn_kv8_copy_pages(const gdn_kv8_pool* p, uint8_t* codes, float* scales,
                              const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
  const gdn_status s = validate_pool(p);
  if (s != GDN_OK) return s;
  if (n < 0) return GDN_ERR_INVALID_ARG;
  if (n == 0 || p->pages == 0) return GDN_OK;
  if (!codes || !scales || !src || !dst) return GDN_ERR_INVALID_ARG;
  if (misaligned({codes}, 15) || misaligned({scales, src, dst}, 3)) return GDN_ERR_MISALIGNED;
  return launch_move(*p, codes, scales, src, dst, nullptr, n, n, false, (cudaStream_t)stream);
}

gdn_status gdn_kv8_fork(const gdn_kv8_pool* p, uint8_t* codes, float* scales, const int32_t* table,
                        const int32_t* lengths, const int32_t* refs, const int32_t* parents,
                        const uint8_t* drop, int32_t* table_out, int32_t* lengths_out,
                        int32_t* refs_out, int32_t* missing, void* workspace,
                        size_t workspace_bytes, void* stream) {
  gdn_status s = validate_pool(p);
  if (s != GDN_OK) return s;
  if (!lengths || !lengths_out || !missing || (!parents == !drop)) return GDN_ERR_INVALID_ARG;
  if (p->cols > 0 && (!table || !table_out)) return GDN_ERR_INVALID_ARG;
  if (p->pages > 0 && (!codes || !scales || !refs || !refs_out)) return GDN_ERR_INVALID_ARG;
  if (misaligned({codes, workspace}, 15) ||
      misaligned({scales, table, lengths, refs, parents, table_out, lengths_out, refs_out, missing}, 3))
    return GDN_ERR_MISALIGNED;
  if (table == table_out || lengths == lengths_out || (refs && refs == refs_out))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < gdn_kv8_pool_workspace_bytes(p))
    return GDN_ERR_WORKSPACE_TOO_SMALL;
  PlanParams q = {};
  q.table = table, q.lengths = lengths, q.refs = refs, q.parents = parents, q.drop = drop;
  q.table_out = table_out, q.lengths_out = lengths_out, q.refs_out = refs_out, q.count_out = missing;
  s = run_plan(kFork, *p, q, workspace, (cudaStream_t)stream);
  if (s != GDN_OK || drop) return s;  // rows that keep or lose their sequence copy nothing
  int32_t* w = static_cast<int32_t*>(workspace);
  return launch_move(*p, codes, scales, w + 4, w + 4 + move_ints(*p), w, 0, p->rows, true,
                     (cudaStream_t)stream);
}

gdn_status gdn_kv8_reserve(const gdn_kv8_pool* p, const int32_t* table, const int32_t* lengths,
                           const int32_t* refs, const int32_t* extra, int32_t* table_out,
                           int32_t* lengths_out, int32_t* refs_out, int32_t* missing,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const gdn_status s = validate_pool(p);
  if (s != GDN_OK) return s;
  if (!lengths || !extra || !lengths_out || !missing) return GDN_ERR_INVALID_ARG;
  if (p->cols > 0 && (!table || !table_out)) return GDN_ERR_INVALID_ARG;
  if (p->pages > 0 && (!refs || !refs_out)) return GDN_ERR_INVALID_ARG;
  if (misaligned({workspace}, 15) ||
      misaligned({table, lengths, refs, extra, table_out, lengths_out, refs_out, missing}, 3))
    return GDN_ERR_MISALIGNED;
  if (table == table_out || lengths == lengths_out || (refs && refs == refs_out))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < gdn_kv8_pool_workspace_bytes(p))
    return GDN_ERR_WORKSPACE_TOO_SMALL;
  PlanParams q = {};
  q.table = table, q.lengths = lengths, q.refs = refs, q.extra = extra;
  q.table_out = table_out, q.lengths_out = lengths_out, q.refs_out = refs_out, q.count_out = missing;
  return run_plan(kReserve, *p, q, workspace, (cudaStream_t)stream);
}

gdn_status gdn_kv8_compact(const gdn_kv8_pool* p, uint8_t* codes, float* scales,
                           const int32_t* table, const int32_t* lengths, const int32_t* refs,
                           int32_t* table_out, int32_t* refs_out, int32_t* live, void* workspace,
                           size_t workspace_bytes, void* stream) {
  gdn_status s = validate_pool(p);
  if (s != GDN_OK) return s;
  if (!lengths || !live) return GDN_ERR_INVALID_ARG;
  if (p->cols > 0 && (!table || !table_out)) return GDN_ERR_INVALID_ARG;
  if (p->pages > 0 && (!codes || !scales || !refs || !refs_out)) return GDN_ERR_INVALID_ARG;
  if (misaligned({codes, workspace}, 15) ||
      misaligned({scales, table, lengths, refs, table_out, refs_out, live}, 3))
    return GDN_ERR_MISALIGNED;
  if (table == table_out || (refs && refs == refs_out)) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < gdn_kv8_pool_workspace_bytes(p))
    return GDN_ERR_WORKSPACE_TOO_SMALL;
  PlanParams q = {};
  q.table = table, q.lengths = lengths, q.refs = refs;
  q.table_out = table_out, q.refs_out = refs_out, q.count_out = live;
  s = run_plan(kCompact, *p, q, workspace, (cudaStream_t)stream);
  if (s != GDN_OK) return s;
  int32_t* w = static_cast<int32_t*>(workspace);
  return launch_move(*p, codes, scales, w + 4, w + 4 + move_ints(*p), w, 0, p->pages / 2, true,
                     (cudaStream_t)stream);
}

}  // extern "C"
