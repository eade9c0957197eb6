// pages.cu — the pages of a paged cache, managed on the device: forks
// (lrkv_pages_fork), room for new rows with copies on write
// (lrkv_pages_extend) and compaction (lrkv_pages_compact).
//
// Tables, lengths and reference counts are small; what a call costs is its
// passes over them, one after the other, and the launches.  So a plan is one
// launch of one cluster of CTAs that goes through its passes with cluster
// barriers between them, the counts of its CTAs exchanged through distributed
// shared memory.  Pages are numbered by prefix sums in a fixed order (the k-th
// free page, the k-th page to move), never by an atomic counter; atomics only
// add and take maxima of integers, whose results do not depend on the order.
//
// The pages that a plan copies are then moved by lrkv_pages_copy_kernel, bound by
// memory: a warp per 2 KB segment of a page of a pool.  It reads how many
// there are from the workspace, so the host never waits.
//
// Measured on GB300, back-to-back calls of a graph: a fork of 64 x 64 blocks 4.4 us,
// of 512 x 512 blocks 9.2 us; room for one more row of 256 sequences, four to a
// prompt, whose begun pages are copied (39 MB of an 8-bit cache), 16.7 us, of which
// the copies' bytes are 6; a compaction that moves 1,067 pages of 426 KB (909 MB
// read and written) 147 us, 0.93 of a measured copy's rate.  The plans are bound
// by latency: each pass waits for the loads of the one before.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <map>
#include <mutex>

#include "decode_plan.h"
#include "host_cache.h"
#include "lrkv.h"
#include "ptx.cuh"
#include "trace.h"

namespace cg = cooperative_groups;

namespace lrkv {

namespace {

constexpr int kPgThreads = 1024, kPgWarps = kPgThreads / 32;
constexpr int kPgMaxCluster = 8, kPgForkCluster = 16;  // CTAs of a plan; of a fork, where the device allows it
constexpr int kPgSegment = 2048;       // bytes of a page that a warp moves at a time
constexpr int kPgCopyThreads = 256;

struct PagesArgs {
  int B, nb, shift, pages;             // sequences, blocks of a table row, log2 of the page size, pages
  const int32_t *table, *lens, *refs;
  int32_t *table_out, *lens_out, *refs_out;
  const int32_t *parent, *keep;        // fork
  const int32_t* new_lens;             // extend
  int32_t* missing;                    // extend, or NULL
  int32_t *moved, *live;               // compact, or NULL
  int copies_follow;                   // 1: the next launch is lrkv_pages_copy_kernel
  // workspace: the status word, how many pages to copy, and arrays
  uint32_t* status;
  int* count;
  int* ws_lens;   // [B]
  int* ws_table;  // [B][nb]
  int* ws_a;      // [pages]
  int* ws_b;      // [pages]
  int* ws_c;      // [pages]
  int4* copies;   // [min(pages, ...)]: from, to, rows
};

struct PoolArgs {
  unsigned char* data;
  long long page_bytes;
  int rows, bytes;      // a piece of `bytes` bytes for every `rows` rows
  int first;            // the pool's first segment among a page's
  int vec;              // bytes of a load: 16 or 4
};
struct CopyArgs {
  PoolArgs pool[LRKV_MAX_POOLS];
  int n, segments;      // pools; segments of a page in all of them
  const int* count;
  const int4* copies;
};

__device__ __forceinline__ int warp_scan(int v) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}
// Exclusive prefix over the CTA's threads; total receives the CTA's sum.
__device__ __forceinline__ int block_prefix(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int incl = warp_scan(v);
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int w = warp_scan(lane < kPgWarps ? s_warp[lane] : 0);
  total = __shfl_sync(0xffffffffu, w, kPgWarps - 1);
  return incl - v + __shfl_sync(0xffffffffu, w, warp) - s_warp[warp];
}
// Sum of the CTAs' values before this one's, and of all; `slot` is this
// exchange's own.  Passes a cluster barrier.
__device__ __forceinline__ int cluster_prefix(cg::cluster_group& cl, int value, int* slot, int& total) {
  if (threadIdx.x == 0) *slot = value;
  cl.sync();
  int before = 0;
  total = 0;
  for (unsigned r = 0; r < cl.num_blocks(); ++r) {
    const int v = *cl.map_shared_rank(slot, r);
    if (r < cl.block_rank()) before += v;
    total += v;
  }
  return before;
}
__device__ __forceinline__ int clamp_len(const PagesArgs& A, int len, bool& bad) {
  const long long cap = static_cast<long long>(A.nb) << A.shift;
  if (len < 0 || len > cap) bad = true;
  return static_cast<int>(min(max(static_cast<long long>(len), 0ll), cap));
}
__device__ __forceinline__ int blocks_of(const PagesArgs& A, int len) {
  return (len >> A.shift) + ((len & ((1 << A.shift) - 1)) != 0);
}
// f(sequence, first block, blocks) for pieces of the tables' rows, a warp each.
constexpr int kPgPiece = 256;
template <typename F>
__device__ __forceinline__ void for_rows(cg::cluster_group& cl, const PagesArgs& A, F f) {
  const int pieces = (A.nb + kPgPiece - 1) / kPgPiece, all = A.B * pieces;
  for (int u = cl.block_rank() * kPgWarps + (threadIdx.x >> 5); u < all; u += cl.num_blocks() * kPgWarps) {
    const int b = u / pieces, j = (u - b * pieces) * kPgPiece;
    f(b, j, min(kPgPiece, A.nb - j));
  }
}
// The status word was cleared before a cluster barrier that every CTA has passed.
__device__ __forceinline__ void add_status(const PagesArgs& A, bool bad, uint32_t more) {
  if (__syncthreads_or(bad)) more |= kDevBounds;
  if (threadIdx.x == 0 && more) atomicOr(A.status, more);
}
// A warp's contiguous share of the pages, a multiple of 32.
__device__ __forceinline__ void page_share(cg::cluster_group& cl, const PagesArgs& A, int& lo, int& hi) {
  const int warps = static_cast<int>(cl.num_blocks()) * kPgWarps;
  const int each = ((A.pages + warps - 1) / warps + 31) / 32 * 32;
  const long long at = static_cast<long long>(cl.block_rank() * kPgWarps + (threadIdx.x >> 5)) * each;
  lo = static_cast<int>(min(at, static_cast<long long>(A.pages)));
  hi = static_cast<int>(min(at + each, static_cast<long long>(A.pages)));
}

}  // namespace

// ===================================================================== fork
__global__ void __launch_bounds__(kPgThreads) lrkv_pages_fork_kernel(const __grid_constant__ PagesArgs A) {
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int at = cl.block_rank() * kPgThreads + threadIdx.x, step = cl.num_blocks() * kPgThreads;
  const bool in_place = A.table_out == A.table;
  bool bad = false;
  pdl_wait();  // the launch before
  if (at == 0) *A.status = 0u;
  if (A.refs_out != A.refs)
    for (int p = at; p < A.pages; p += step) A.refs_out[p] = A.refs[p];
  // the length of sequence b after the call
  auto length = [&](int b, int& parent) {
    parent = A.parent ? A.parent[b] : b;
    const int keep = A.keep ? A.keep[b] : INT_MAX;
    int len = 0;
    if (parent >= 0 && parent < A.B) len = clamp_len(A, A.lens[parent], bad);
    else if (parent != -1) bad = true;
    if (keep < 0) bad = true;
    return min(len, max(keep, 0));
  };
  for (int b = at; b < A.B; b += step) {
    int parent;
    A.ws_lens[b] = length(b, parent);
  }
  cl.sync();
  int32_t* to = in_place ? A.ws_table : A.table_out;
  for_rows(cl, A, [&](int b, int j0, int n) {
    int parent;
    const int want = blocks_of(A, length(b, parent)), used = blocks_of(A, clamp_len(A, A.lens[b], bad));
    const int32_t* mine = A.table + static_cast<long long>(b) * A.nb;
    const int32_t* from = A.table + static_cast<long long>(max(parent, 0)) * A.nb;
    int32_t* row = to + static_cast<long long>(b) * A.nb;
    constexpr int kEach = kPgPiece / 32;
    int before[kEach], after[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = j0 + lane + 32 * i;
      before[i] = j < j0 + n && j < used ? mine[j] : -1;
      after[i] = j < j0 + n && j < want ? from[j] : -1;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = j0 + lane + 32 * i;
      if (j >= j0 + n) continue;
      row[j] = after[i];
      const bool was = static_cast<unsigned>(before[i]) < static_cast<unsigned>(A.pages);
      const bool is = static_cast<unsigned>(after[i]) < static_cast<unsigned>(A.pages);
      if ((j < used && !was) || (j < want && !is)) bad = true;
      if (before[i] == after[i]) continue;
      if (was) atomicSub(&A.refs_out[before[i]], 1);
      if (is) atomicAdd(&A.refs_out[after[i]], 1);
    }
  });
  cl.sync();
  if (in_place)
    for (long long e = at; e < static_cast<long long>(A.B) * A.nb; e += step) A.table_out[e] = A.ws_table[e];
  for (int b = at; b < A.B; b += step) A.lens_out[b] = A.ws_lens[b];
  add_status(A, bad, 0u);
}

// =================================================================== extend
// ws_a, ws_b: of a shared page that new rows begin inside of, how many sequences
// do so and the last of them; ws_c: the k-th free page.
__global__ void __launch_bounds__(kPgThreads) lrkv_pages_extend_kernel(const __grid_constant__ PagesArgs A) {
  extern __shared__ int s_dyn[];
  __shared__ int s_warp[kPgWarps], s_free[kPgWarps], s_slot;
  int* s_len = s_dyn;            // [B] lengths
  int* s_new = s_len + A.B;      // [B] lengths after the call
  int* s_page = s_new + A.B;     // [B] the begun page that is copied, or -1
  int* s_first = s_page + A.B;   // [B] place of the first page taken
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at = cl.block_rank() * kPgThreads + tid, step = cl.num_blocks() * kPgThreads;
  const int rest = (1 << A.shift) - 1;
  pdl_wait();  // the launch before
  if (A.copies_follow) pdl_trigger();  // (they wait for this grid; any other launch starts when it has ended)
  bool bad = false;
  if (at == 0) *A.status = 0u;
  // 1. lengths; the page that a sequence's new rows begin inside of, if others use it too (each CTA for itself)
  int shared = 0;
  for (int b = tid; b < A.B; b += kPgThreads) {
    const int len = clamp_len(A, A.lens[b], bad), to = max(len, clamp_len(A, A.new_lens[b], bad));
    int page = -1;
    if (to > len && (len & rest) != 0) {
      page = A.table[static_cast<long long>(b) * A.nb + (len >> A.shift)];
      if (page < 0 || page >= A.pages) {
        bad = true;
        page = -1;
      } else if (A.refs[page] > 1) {
        A.ws_a[page] = 0;
        A.ws_b[page] = -1;
        shared = 1;
      } else {
        page = -1;
      }
    }
    s_len[b] = len;
    s_new[b] = to;
    s_page[b] = page;
  }
  // meanwhile: the free pages of each warp's share, and copies of what has outputs of its own
  int lo, hi, mine = 0;
  page_share(cl, A, lo, hi);
#pragma unroll 4
  for (int p = lo + lane; p < hi; p += 32) {
    const int refs = A.refs[p];
    mine += refs <= 0;
    if (A.refs_out != A.refs) A.refs_out[p] = refs;
  }
  const long long entries = static_cast<long long>(A.B) * A.nb;
  if (A.table_out != A.table)
#pragma unroll 4
    for (long long e = at; e < entries; e += step) A.table_out[e] = A.table[e];
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) s_free[warp] = mine;
  shared = __syncthreads_or(shared);  // (the same in every CTA)
  if (shared) {
    cl.sync();
    if (cl.block_rank() == 0)
      for (int b = tid; b < A.B; b += kPgThreads)
        if (s_page[b] >= 0) {
          atomicAdd(&A.ws_a[s_page[b]], 1);
          atomicMax(&A.ws_b[s_page[b]], b);
        }
  }
  const int incl = warp_scan(lane < kPgWarps ? s_free[lane] : 0);
  int free_pages;
  const int before = cluster_prefix(cl, __shfl_sync(0xffffffffu, incl, kPgWarps - 1), &s_slot, free_pages);
  // 2. what every sequence takes (each CTA for itself); the pages copied, in order
  int total = 0, copied = 0;
  for (int b0 = 0; b0 < A.B; b0 += kPgThreads) {
    const int b = b0 + tid;
    int need = 0, copy = 0;
    if (b < A.B) {
      const int page = s_page[b];
      need = blocks_of(A, s_new[b]) - blocks_of(A, s_len[b]);
      if (page >= 0) {
        // (of the users of a page that all write, the last one keeps it)
        copy = !(A.refs[page] == __ldcg(A.ws_a + page) && b == __ldcg(A.ws_b + page));
        if (!copy) s_page[b] = -1;
      }
      need += copy;
    }
    int sum, sum_copies;
    const int first = block_prefix(need, s_warp, sum), nth = block_prefix(copy, s_warp, sum_copies);
    if (b < A.B) s_first[b] = total + first;
    if (copy && cl.block_rank() == 0)  // (the page to copy to is not known yet: its place among the taken)
      A.copies[copied + nth] = make_int4(s_page[b], total + first, s_len[b] & rest, 0);
    total += sum;
    copied += sum_copies;
  }
  // 3. the free pages in order, as many as are taken
  int rank = before + __shfl_sync(0xffffffffu, incl, warp) - s_free[warp];
  for (int p0 = lo; p0 < hi && rank < total; p0 += 32) {
    const bool is = p0 + lane < hi && A.refs[p0 + lane] <= 0;
    const unsigned m = __ballot_sync(0xffffffffu, is);
    const int k = rank + __popc(m & ((1u << lane) - 1u));
    if (is && k < total) A.ws_c[k] = p0 + lane;
    rank += __popc(m);
  }
  cl.sync();
  // 4. hand them out, if there are enough
  const bool enough = total <= free_pages;
  if (enough) {
    for (int k = at; k < total; k += step) A.refs_out[__ldcg(A.ws_c + k)] = 1;
    for (int b = cl.block_rank() * kPgWarps + warp; b < A.B; b += cl.num_blocks() * kPgWarps) {
      const int copy = s_page[b] >= 0, have = blocks_of(A, s_len[b]), want = blocks_of(A, s_new[b]);
      int32_t* row = A.table_out + static_cast<long long>(b) * A.nb;
      if (copy && lane == 0) {
        row[s_len[b] >> A.shift] = __ldcg(A.ws_c + s_first[b]);
        atomicSub(&A.refs_out[s_page[b]], 1);
      }
      for (int j = have + lane; j < want; j += 32) row[j] = __ldcg(A.ws_c + s_first[b] + copy + j - have);
      if (lane == 0) A.lens_out[b] = s_new[b];
    }
    if (cl.block_rank() == 0)
      for (int k = tid; k < copied; k += kPgThreads) A.copies[k].y = __ldcg(A.ws_c + A.copies[k].y);
  } else {
    for (int b = at; b < A.B; b += step) A.lens_out[b] = A.lens[b];
  }
  if (at == 0) {
    *A.count = enough ? copied : 0;
    if (A.missing) *A.missing = enough ? 0 : total - free_pages;
  }
  add_status(A, bad, enough ? 0u : kDevNoPages);
}

// ================================================================== compact
// ws_a: the k-th free page below the end; ws_b: every page's new number; ws_c:
// the k-th used page.
__global__ void __launch_bounds__(kPgThreads) lrkv_pages_compact_kernel(const __grid_constant__ PagesArgs A) {
  __shared__ int s_live[kPgWarps], s_slot;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at = cl.block_rank() * kPgThreads + tid, step = cl.num_blocks() * kPgThreads;
  pdl_wait();  // the launch before
  if (A.copies_follow) pdl_trigger();  // (they wait for this grid; any other launch starts when it has ended)
  bool bad = false;
  if (at == 0) *A.status = 0u;
  // 1. how many pages are in use: they go to the pages before that number
  int lo, hi, mine = 0;
  page_share(cl, A, lo, hi);
#pragma unroll 4
  for (int p = lo + lane; p < hi; p += 32) mine += A.refs[p] > 0;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) s_live[warp] = mine;
  __syncthreads();
  const int incl = warp_scan(lane < kPgWarps ? s_live[lane] : 0);
  int live;
  const int before = cluster_prefix(cl, __shfl_sync(0xffffffffu, incl, kPgWarps - 1), &s_slot, live);
  // 2. numbers of the used pages and of the free ones before the end: a page p there has p less the used ones
  // before it.  (*count: used pages before the end, for the moment)
  int used = before + __shfl_sync(0xffffffffu, incl, warp) - s_live[warp];
  for (int p0 = lo; p0 < hi; p0 += 32) {
    const int p = p0 + lane;
    const bool is = p < hi && A.refs[p] > 0;
    const unsigned m = __ballot_sync(0xffffffffu, is);
    const int rank = used + __popc(m & ((1u << lane) - 1u));
    if (p < hi) {
      if (is) A.ws_c[rank] = p;
      else if (p < live) A.ws_a[p - rank] = p;
      A.ws_b[p] = is && p < live ? p : -1;
      if (p == live) *A.count = rank;
    }
    used += __popc(m);
  }
  if (at == 0 && live == A.pages) *A.count = live;
  cl.sync();
  const int low = __ldcg(A.count), moves = live - low;
  // 3. the k-th used page past the end into the k-th free one before it, with its references
  for (int k = at; k < moves; k += step) {
    const int from = __ldcg(A.ws_c + low + k), to = __ldcg(A.ws_a + k);
    A.copies[k] = make_int4(from, to, 1 << A.shift, 0);
    A.ws_b[from] = to;
    A.refs_out[to] = A.refs[from];
  }
  if (A.refs_out != A.refs)
    for (int k = at; k < low; k += step) {
      const int p = __ldcg(A.ws_c + k);
      A.refs_out[p] = A.refs[p];
    }
  cl.sync();
  // 4. nothing lies past the end any more; tables
  for (int p = live + at; p < A.pages; p += step) A.refs_out[p] = 0;
  if (A.moved)
    for (int p = at; p < A.pages; p += step) A.moved[p] = __ldcg(A.ws_b + p);
  for_rows(cl, A, [&](int b, int j0, int n) {
    const int in_use = blocks_of(A, clamp_len(A, A.lens[b], bad));
    const int32_t* from = A.table + static_cast<long long>(b) * A.nb;
    int32_t* row = A.table_out + static_cast<long long>(b) * A.nb;
    constexpr int kEach = kPgPiece / 32;
    int page[kEach], to[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = j0 + lane + 32 * i;
      page[i] = j < j0 + n ? from[j] : -1;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = j0 + lane + 32 * i;
      to[i] = j < j0 + n && j < in_use && static_cast<unsigned>(page[i]) < static_cast<unsigned>(A.pages)
                  ? __ldcg(A.ws_b + page[i])
                  : -1;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = j0 + lane + 32 * i;
      if (j >= j0 + n) continue;
      if (j < in_use && to[i] < 0) bad = true;
      row[j] = to[i] >= 0 ? to[i] : page[i];
    }
  });
  if (at == 0) {
    *A.count = moves;
    if (A.live) *A.live = live;
  }
  add_status(A, bad, 0u);
}

// =================================================================== copies
__global__ void __launch_bounds__(kPgCopyThreads) lrkv_pages_copy_kernel(const __grid_constant__ CopyArgs A) {
  pdl_wait();  // the plan
  const int lane = threadIdx.x & 31;
  const long long all = static_cast<long long>(*A.count) * A.segments;
  const long long step = static_cast<long long>(gridDim.x) * (kPgCopyThreads / 32);
  for (long long t = static_cast<long long>(blockIdx.x) * (kPgCopyThreads / 32) + (threadIdx.x >> 5); t < all;
       t += step) {
    const int c = static_cast<int>(t / A.segments), s = static_cast<int>(t - static_cast<long long>(c) * A.segments);
    const int4 copy = __ldg(A.copies + c);
    int i = 0;
    while (i + 1 < A.n && A.pool[i + 1].first <= s) ++i;
    const PoolArgs& P = A.pool[i];
    const long long bytes = static_cast<long long>((copy.z + P.rows - 1) / P.rows) * P.bytes;
    const long long off = static_cast<long long>(s - P.first) * kPgSegment;
    if (off >= bytes) continue;
    const int n = static_cast<int>(min(bytes - off, static_cast<long long>(kPgSegment)));
    const unsigned char* from = P.data + copy.x * P.page_bytes + off;
    unsigned char* to = P.data + copy.y * P.page_bytes + off;
    if (P.vec == 16) {
      uint4 v[kPgSegment / 512];
#pragma unroll
      for (int k = 0; k < kPgSegment / 512; ++k)
        if (16 * (lane + 32 * k) < n) v[k] = *reinterpret_cast<const uint4*>(from + 16 * (lane + 32 * k));
#pragma unroll
      for (int k = 0; k < kPgSegment / 512; ++k)
        if (16 * (lane + 32 * k) < n) *reinterpret_cast<uint4*>(to + 16 * (lane + 32 * k)) = v[k];
    } else {
      uint32_t v[kPgSegment / 128];
#pragma unroll
      for (int k = 0; k < kPgSegment / 128; ++k)
        if (4 * (lane + 32 * k) < n) v[k] = *reinterpret_cast<const uint32_t*>(from + 4 * (lane + 32 * k));
#pragma unroll
      for (int k = 0; k < kPgSegment / 128; ++k)
        if (4 * (lane + 32 * k) < n) *reinterpret_cast<uint32_t*>(to + 4 * (lane + 32 * k)) = v[k];
    }
  }
}

// ======================================================================= host
namespace {

lrkv_status pages_check(int batch, int max_blocks, int page_size, int num_pages) {
  if (batch < 1 || max_blocks < 1 || num_pages < 1) return LRKV_ERR_INVALID_ARG;
  if (page_size < 16 || (page_size & (page_size - 1)) != 0) return LRKV_ERR_INVALID_ARG;
  constexpr long long most = 1ll << 30;
  if (batch > kMaxBatch || static_cast<long long>(batch) * max_blocks > most || num_pages > most ||
      static_cast<long long>(max_blocks) * page_size > (1ll << 31) - 1)
    return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// status, count | ws_lens | ws_table | ws_a | ws_b | ws_c | copies
size_t pages_bytes(int B, int nb, int pages) {
  return 256 + up(4ull * B) + up(4ull * B * nb) + 3 * up(4ull * pages) +
         up(sizeof(int4) * static_cast<size_t>(std::max(B, pages)));
}

void pages_bind(PagesArgs& A, void* ws) {
  unsigned char* p = static_cast<unsigned char*>(ws);
  A.status = reinterpret_cast<uint32_t*>(p);
  A.count = reinterpret_cast<int*>(p + 16);
  p += 256;
  A.ws_lens = reinterpret_cast<int*>(p);
  p += up(4ull * A.B);
  A.ws_table = reinterpret_cast<int*>(p);
  p += up(4ull * A.B * A.nb);
  A.ws_a = reinterpret_cast<int*>(p);
  p += up(4ull * A.pages);
  A.ws_b = reinterpret_cast<int*>(p);
  p += up(4ull * A.pages);
  A.ws_c = reinterpret_cast<int*>(p);
  p += up(4ull * A.pages);
  A.copies = reinterpret_cast<int4*>(p);
}

// Checks and fields that the three calls share.
lrkv_status pages_args(PagesArgs& A, int batch, int max_blocks, int page_size, int num_pages, const int32_t* table,
                       const int32_t* lens, const int32_t* refs, int32_t* table_out, int32_t* refs_out, void* ws,
                       size_t ws_bytes) {
  const lrkv_status st = pages_check(batch, max_blocks, page_size, num_pages);
  if (st != LRKV_OK) return st;
  if (!table || !lens || !refs || !table_out || !refs_out) return LRKV_ERR_INVALID_ARG;
  if (!ws) return LRKV_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0) return LRKV_ERR_INVALID_ARG;
  if (ws_bytes < pages_bytes(batch, max_blocks, num_pages)) return LRKV_ERR_WORKSPACE;
  A = PagesArgs{};
  A.B = batch; A.nb = max_blocks; A.pages = num_pages;
  while ((1 << A.shift) < page_size) ++A.shift;
  A.table = table; A.lens = lens; A.refs = refs;
  A.table_out = table_out; A.refs_out = refs_out;
  pages_bind(A, ws);
  return LRKV_OK;
}

// Whether a cluster of kPgForkCluster CTAs of a fork (more than the portable 8: the kernel's opt-in is set here) can
// run on the current device.
bool fork_cluster_fits() {
  static std::mutex mu;
  static std::map<int, bool> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lock(mu);
  const auto it = known.find(dev);
  if (it != known.end()) return it->second;
  const void* kern = reinterpret_cast<const void*>(&lrkv_pages_fork_kernel);
  int n = 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPgForkCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPgForkCluster);
  cfg.blockDim = dim3(kPgThreads);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool fits = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n >= 1;
  if (!fits) cudaGetLastError();  // (eight are used then)
  known[dev] = fits;
  return fits;
}

// One CTA for the smallest tables, where its barriers are the cheapest.  (One against eight CTAs: 5.9 and 4.4 us for a
// fork of 64 x 64 blocks, 59 and 12.3 us for 512 x 512 with prompts in common.)  Sixteen for a fork, whose passes share
// the table out (12.3 and 9.2 us for 512 x 512); not for the others, whose passes over the sequences every CTA makes
// for itself (an extension for 256 more rows took 1.3 us longer).
template <typename K>
lrkv_status pages_launch(K kern, const PagesArgs& A, int most, size_t smem, cudaStream_t stream) {
  const long long work = static_cast<long long>(A.B) * A.nb + A.pages;
  int n = 1;
  while (n < most && work > 1024ll * n) n *= 2;
  if (smem > 32 * 1024 &&  // (with the static part it may pass 48 KB)
      ensure_kernel_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem)) != cudaSuccess)
    return LRKV_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  // (launched ahead of the end of the launch before, for which it waits: 0.2 to 0.4 us less of every call in a graph,
  // 17.1 -> 16.7 for 256 more rows; one by one from Python 20.5 -> 18.4 to 19.8 there, 149-152 -> 145-147 for 4,269
  // pages, nothing where the host is the bound)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n);
  cfg.blockDim = dim3(kPgThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, A) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

lrkv_status copy_args(CopyArgs& C, PagesArgs& A, const lrkv_pool* pools, int n) {
  if (n < 0 || n > LRKV_MAX_POOLS || (n > 0 && !pools)) return LRKV_ERR_INVALID_ARG;
  C = CopyArgs{};
  C.n = n;
  long long segments = 0;
  for (int i = 0; i < n; ++i) {
    const lrkv_pool& p = pools[i];
    if (!p.data || p.bytes < 1 || p.bytes % 4 != 0 || (reinterpret_cast<uintptr_t>(p.data) & 3u) != 0 || p.rows < 1 ||
        p.rows > (1 << A.shift) || (1 << A.shift) % p.rows != 0)
      return LRKV_ERR_INVALID_ARG;
    PoolArgs& P = C.pool[i];
    P.data = static_cast<unsigned char*>(p.data);
    P.rows = p.rows;
    P.bytes = p.bytes;
    P.page_bytes = static_cast<long long>((1 << A.shift) / p.rows) * p.bytes;
    P.vec = p.bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(p.data) & 15u) == 0 ? 16 : 4;
    P.first = static_cast<int>(segments);
    segments += (P.page_bytes + kPgSegment - 1) / kPgSegment;
    if (segments > (1 << 30)) return LRKV_ERR_UNSUPPORTED;
  }
  C.segments = static_cast<int>(segments);
  A.copies_follow = n > 0;
  C.count = A.count;
  C.copies = A.copies;
  return LRKV_OK;
}

lrkv_status copy_launch(const CopyArgs& C, int sms, cudaStream_t stream) {
  if (C.n == 0) return LRKV_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms * (2048 / kPgCopyThreads));
  cfg.blockDim = dim3(kPgCopyThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lrkv_pages_copy_kernel, C) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

}  // namespace

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_pages_workspace_size(int batch, int max_blocks, int num_pages, size_t* bytes) {
  if (!bytes) return LRKV_ERR_INVALID_ARG;
  const lrkv_status st = lrkv::pages_check(batch, max_blocks, 16, num_pages);
  if (st != LRKV_OK) return st;
  *bytes = lrkv::pages_bytes(batch, max_blocks, num_pages);
  return LRKV_OK;
}

lrkv_status lrkv_pages_fork(int batch, int max_blocks, int page_size, int num_pages, const int32_t* parent,
                            const int32_t* keep, const int32_t* block_table, const int32_t* seq_lens,
                            const int32_t* refs, int32_t* table_out, int32_t* lens_out, int32_t* refs_out, void* ws,
                            size_t ws_bytes, lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_pages_fork");
  lrkv::PagesArgs A;
  if (!lens_out) return LRKV_ERR_INVALID_ARG;
  const lrkv_status st = lrkv::pages_args(A, batch, max_blocks, page_size, num_pages, block_table, seq_lens, refs,
                                          table_out, refs_out, ws, ws_bytes);
  if (st != LRKV_OK) return st;
  A.lens_out = lens_out;
  A.parent = parent;
  A.keep = keep;
  return lrkv::pages_launch(lrkv::lrkv_pages_fork_kernel, A,
                            lrkv::fork_cluster_fits() ? lrkv::kPgForkCluster : lrkv::kPgMaxCluster, 0,
                            static_cast<cudaStream_t>(stream));
}

lrkv_status lrkv_pages_extend(int batch, int max_blocks, int page_size, int num_pages, const int32_t* new_lens,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* refs,
                              int32_t* table_out, int32_t* lens_out, int32_t* refs_out, int32_t* missing,
                              const lrkv_pool* pools, int n_pools, void* ws, size_t ws_bytes, lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_pages_extend");
  lrkv::PagesArgs A;
  if (!new_lens || !lens_out) return LRKV_ERR_INVALID_ARG;
  lrkv_status st = lrkv::pages_args(A, batch, max_blocks, page_size, num_pages, block_table, seq_lens, refs,
                                    table_out, refs_out, ws, ws_bytes);
  if (st != LRKV_OK) return st;
  A.lens_out = lens_out;
  A.new_lens = new_lens;
  A.missing = missing;
  lrkv::CopyArgs C;
  if ((st = lrkv::copy_args(C, A, pools, n_pools)) != LRKV_OK) return st;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  if ((st = lrkv::pages_launch(lrkv::lrkv_pages_extend_kernel, A, lrkv::kPgMaxCluster,
                               4 * sizeof(int) * static_cast<size_t>(batch), static_cast<cudaStream_t>(stream))) !=
      LRKV_OK)
    return st;
  return lrkv::copy_launch(C, sms, static_cast<cudaStream_t>(stream));
}

lrkv_status lrkv_pages_compact(int batch, int max_blocks, int page_size, int num_pages, const int32_t* block_table,
                               const int32_t* seq_lens, const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                               int32_t* moved, int32_t* live, const lrkv_pool* pools, int n_pools, void* ws,
                               size_t ws_bytes, lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_pages_compact");
  lrkv::PagesArgs A;
  lrkv_status st = lrkv::pages_args(A, batch, max_blocks, page_size, num_pages, block_table, seq_lens, refs,
                                    table_out, refs_out, ws, ws_bytes);
  if (st != LRKV_OK) return st;
  A.moved = moved;
  A.live = live;
  lrkv::CopyArgs C;
  if ((st = lrkv::copy_args(C, A, pools, n_pools)) != LRKV_OK) return st;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  if ((st = lrkv::pages_launch(lrkv::lrkv_pages_compact_kernel, A, lrkv::kPgMaxCluster, 0,
                               static_cast<cudaStream_t>(stream))) != LRKV_OK)
    return st;
  return lrkv::copy_launch(C, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
