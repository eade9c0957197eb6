// evict.cu — eviction from the factored cache by accumulated attention
// weight (lrkv_evict): the rows of a sequence that gathered least go, so that
// at most `budget` stay.
//
// A sequence of L rows keeps n = min(L, budget) of them: the held rows (the
// oldest `sink` and the newest `recent` tokens) and the heaviest others,
// equal weights by the lower row.  The shared row belongs to every head, so a
// token goes for all heads at once and its weight is the sum over them.
//
// Attention over a set of rows does not depend on their order, so nothing is
// shifted: a kept row below n stays where it is, and the kept rows at or past
// n (as many as there are dropped rows below n) move into those holes, the
// k-th into the k-th.  That moves the fewest rows there can be, no row is both
// read and written, and all moves run at once.
//
// Measured: 32 x 4097 rows to 4096 22 us a call (the selection's dependent
// passes and the call's own host time); 8 x 9-16K rows to 4096 79 us, 304 MB of
// moves at 5.3 TB/s behind a 22 us selection; 256K rows to 32K 86 us, half of it
// the selection: three cluster-wide counts at ~6.5K cycles each, the rest its
// passes over 16K rows a CTA.
//
// 1. lrkv_evict_select_kernel, one cluster of CTAs per sequence: a radix
//    selection (11 + 11 + 10 bits) of the order-preserving integer image of
//    the weights finds the smallest kept value, each CTA counting its rows in
//    shared memory and the cluster adding the counts up through distributed
//    shared memory; then a bit per row and prefixes over words, warps and the
//    cluster rank equal values, holes and moved rows.
// 2. lrkv_evict_move_kernel copies each moved row: 4 cache tensors (bulk copies
//    through shared memory; through registers, 16 bytes a thread, the same moves
//    ran at 4.2 TB/s), key scales, positions, weight, age.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
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

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;          // 11 bits a level (the last level uses 1024)
constexpr int kEvMaxCluster = 16;      // (more than 8 needs the kernel's opt-in)
constexpr int kEvCacheRows = 40 * 1024;  // rows whose keys a CTA keeps in shared memory
constexpr int kEvUnroll = 4;             // rows a thread has in flight per pass
constexpr int kMoveWarps = 32;           // warps of a moving CTA at most, a slot of shared memory each
constexpr int kMoveSmem = 216 * 1024;    // of the slots
constexpr int kMoveSlotMax = 27 * 1024;  // bytes of a slot at most (longer rows go in parts)
constexpr uint32_t kKeyHeld = 0xffffffffu;  // above every weight's key
constexpr uint32_t kKeyOut = 0u;            // below every weight's key

struct EvictParams {
  int B, max_len, budget, sink, recent;
  int cap;                 // entries of a move list: min(budget, max_len - budget)
  int rows_per_cta;        // rows of one CTA of the cluster (a multiple of 32 * kEvWarps)
  int cached;              // 1: the keys of a CTA's rows are kept in shared memory
  int page_shift, num_pages, max_blocks;
  const int32_t* block_table;  // [B][max_blocks] or NULL
  const int32_t* seq_lens;
  const float* weights;
  const int32_t* order;    // or NULL: a row's age is its index
  float* weights_out;
  int32_t* order_out;      // or NULL
  int32_t* new_lens;
  int32_t* kept;           // [B][budget] or NULL
  // workspace
  uint32_t* status;
  uint32_t* flags;         // [B] status bits of each sequence, written every call
  int32_t* moves;          // [B] moved rows
  int2* src;               // [B][cap] (logical, physical) row of the k-th moved row
  int2* dst;               // [B][cap] (logical, physical) row of the k-th hole
  uint32_t* masks;         // [B][2][ceil(max_len / 32)] row masks (when not in shared memory)
  // moved data
  int slot;                // bytes of a moving warp's slot (a multiple of 128)
  int n16[4];              // 16-byte pieces of a row of each cache tensor
  unsigned char* base[4];
  int H, axes;
  float* key_scale;        // [B][H][max_len] or NULL
  int32_t* positions;      // [B][max_len][axes] or NULL
  long long wait_limit;    // bound of a moving warp's waits for its copies (SM cycles)
};

// Order-preserving image of a weight: larger weight, larger integer, -0 as
// +0 and NaN as -infinity.  Neither kKeyHeld nor kKeyOut is an image.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Adds each lane's bin (where `on`) to a table in shared memory.  Weights tie
// (rows nothing looked at), so the lanes that share the first one's bin are
// added at once; the others add for themselves.  (Grouping all lanes by a
// match instruction took longer than the additions it saved.)
__device__ __forceinline__ void tally(int* hist, bool on, uint32_t bin) {
  const unsigned active = __ballot_sync(0xffffffffu, on);
  if (!active) return;
  const int first = __ffs(active) - 1;
  const uint32_t lead = __shfl_sync(0xffffffffu, bin, first);
  const unsigned same = __ballot_sync(0xffffffffu, on && bin == lead);
  if (on) {
    if (bin != lead) atomicAdd(&hist[bin], 1);
    else if ((threadIdx.x & 31) == first) atomicAdd(&hist[bin], __popc(same));
  }
}

// Exclusive prefix over the CTA's warps of a per-warp count (the same value
// on every lane of a warp); total receives the CTA's sum.
__device__ __forceinline__ int warp_prefix(int count, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) s_warp[warp] = count;
  __syncthreads();
  int v = lane < kEvWarps ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  total = __shfl_sync(0xffffffffu, v, kEvWarps - 1);
  const int mine = __shfl_sync(0xffffffffu, v, warp);
  return mine - count;
}

// The cluster's values of one shared integer: lane c of every warp holds CTA c's
// (c < ncta, at most 16).  One warp fetches them, all remote reads in flight at
// once (every warp for itself took 3K cycles more); s_all is this gather's own.
__device__ __forceinline__ int from_cluster(const cg::cluster_group& cluster, int* value, int ncta, int* s_all) {
  if (threadIdx.x < static_cast<unsigned>(ncta)) s_all[threadIdx.x] = *cluster.map_shared_rank(value, threadIdx.x);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return lane < ncta ? s_all[lane] : 0;
}
__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Physical cache row of logical row t (page * page_size + offset), or -1 when
// the block table names no page of the pool.
__device__ __forceinline__ int physical_row(const EvictParams& P, int b, int t) {
  if (!P.block_table) return b * P.max_len + t;
  const int page = P.block_table[static_cast<size_t>(b) * P.max_blocks + (t >> P.page_shift)];
  if (page < 0 || page >= P.num_pages) return -1;
  return (page << P.page_shift) + (t & ((1 << P.page_shift) - 1));
}

}  // namespace

__global__ void __launch_bounds__(kEvThreads, 1) lrkv_evict_select_kernel(const EvictParams P) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ncta = static_cast<int>(cluster.num_blocks());
  const int b = blockIdx.x / ncta;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ uint32_t s_keys[];          // when cached: [rows_per_cta], then two bits a row
  __shared__ int s_hist[3][kEvBins];            // one table per level: no level waits to clear another's
  __shared__ int s_sum[kEvBins / 2];            // this CTA's share of a level's cluster-wide counts
  __shared__ int s_warp[kEvWarps];
  __shared__ int s_cta[4];                      // this CTA's largest age, held rows, equal rows, holes
  __shared__ int s_cta2;                        // ... moved rows
  __shared__ int s_bin, s_above, s_bad;
  __shared__ int s_all[5][kEvMaxCluster];

  pdl_trigger();
  for (int i = tid; i < 3 * kEvBins; i += kEvThreads) (&s_hist[0][0])[i] = 0;
  if (tid < 4) s_cta[tid] = 0;
  if (tid == 0) s_bad = 0;
  pdl_wait();
  int L = P.seq_lens[b];
  const bool bad_len = L < 0 || L > P.max_len;
  L = min(max(L, 0), P.max_len);
  const int n = min(L, P.budget);
  const float* w = P.weights + static_cast<size_t>(b) * P.max_len;
  const int32_t* age = P.order ? P.order + static_cast<size_t>(b) * P.max_len : nullptr;
  // rows of this CTA, and of this warp: contiguous, a multiple of 32 apart
  const int lo = min(rank * P.rows_per_cta, L), hi = min(lo + P.rows_per_cta, L);
  const int per_warp = P.rows_per_cta / kEvWarps;
  const int wlo = min(lo + warp * per_warp, hi), whi = min(wlo + per_warp, hi);
  __syncthreads();

  int threshold_need = 0;          // rows equal to the threshold that are kept
  uint32_t threshold = kKeyOut;    // smallest kept key
  bool among_held = false;         // more held rows than n: they compete among themselves
  const bool all = L <= n;         // nothing goes
  int newest = L - 1;              // the largest age (one past it need not fit 32 bits)
  auto key = [&](float x, int a) -> uint32_t {  // of weight x and age a
    const uint32_t k = weight_key(x);
    const bool hd = a < P.sink || a > newest - P.recent;
    return among_held ? (hd ? k : kKeyOut) : (hd ? kKeyHeld : k);
  };
  // Keys of rows t, t + 32, ... (kKeyOut past whi; some row of the warp must be
  // below it).  Every load is made, of the last row where there is none: loads
  // behind a condition wait for one another (22K cycles of 16K rows, against 6K).
  auto make_keys = [&](int t, uint32_t (&k)[kEvUnroll]) {
    float x[kEvUnroll];
    int a[kEvUnroll];
#pragma unroll
    for (int u = 0; u < kEvUnroll; ++u) {
      const int at = min(t + 32 * u, whi - 1);
      x[u] = w[at];
      a[u] = age ? age[at] : at;
    }
#pragma unroll
    for (int u = 0; u < kEvUnroll; ++u) k[u] = t + 32 * u < whi ? key(x[u], a[u]) : kKeyOut;
  };
  auto keys_at = [&](int t, uint32_t (&k)[kEvUnroll]) {
    if (P.cached) {
#pragma unroll
      for (int u = 0; u < kEvUnroll; ++u) k[u] = s_keys[min(t + 32 * u, whi - 1) - lo];
#pragma unroll
      for (int u = 0; u < kEvUnroll; ++u) k[u] = t + 32 * u < whi ? k[u] : kKeyOut;
    } else {
      make_keys(t, k);
    }
  };

  if (!all) {
    if (age) {
      int m = 0;
      for (int t = wlo + lane; t < whi; t += 32 * kEvUnroll) {
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u)
          m = max(m, age[min(t + 32 * u, whi - 1)]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) atomicMax(&s_cta[0], m);
      cluster.sync();
      newest = __reduce_max_sync(0xffffffffu, from_cluster(cluster, &s_cta[0], ncta, s_all[0]));
    }
    // keys, and the counts of their highest 11 bits (few bins hold most rows, so
    // neighbouring lanes count in three tables)
    int count = 0;
    for (int t = wlo + lane; t - lane < whi; t += 32 * kEvUnroll) {
      uint32_t k[kEvUnroll];
      make_keys(t, k);
#pragma unroll
      for (int u = 0; u < kEvUnroll; ++u) {
        if (t - lane + 32 * u >= whi) break;
        if (P.cached && t + 32 * u < whi) s_keys[t + 32 * u - lo] = k[u];
        count += k[u] == kKeyHeld;
        tally(s_hist[lane % 3], k[u] != kKeyHeld && k[u] != kKeyOut, k[u] >> 21);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
    if (lane == 0) atomicAdd(&s_cta[1], count);
    __syncthreads();
    for (int i = tid; i < kEvBins; i += kEvThreads) {
      s_hist[0][i] += s_hist[1][i] + s_hist[2][i];
      s_hist[1][i] = s_hist[2][i] = 0;
    }
    cluster.sync();
    int need = n - warp_sum(from_cluster(cluster, &s_cta[1], ncta, s_all[1]));
    if (need < 0) {
      among_held = true;
      need = n;
      // counted again over the held rows alone (every CTA has read the others' first counts)
      cluster.sync();
      for (int i = tid; i < kEvBins; i += kEvThreads) s_hist[0][i] = 0;
      __syncthreads();
      for (int t = wlo + lane; t - lane < whi; t += 32 * kEvUnroll) {
        uint32_t k[kEvUnroll];
        make_keys(t, k);
#pragma unroll
        for (int u = 0; u < kEvUnroll; ++u) {
          if (t - lane + 32 * u >= whi) break;
          if (P.cached && t + 32 * u < whi) s_keys[t + 32 * u - lo] = k[u];
          tally(s_hist[0], k[u] != kKeyOut, k[u] >> 21);
        }
      }
      cluster.sync();
    }
    if (need == 0) {
      threshold = kKeyHeld;  // exactly the held rows
    } else {
      // the need-th largest key, 11 + 11 + 10 bits
      uint32_t prefix = 0;
      int width = 0;
#pragma unroll 1
      for (int level = 0; level < 3; ++level) {
        const int bits = level < 2 ? 11 : 10, shift = 32 - width - bits;
        int* hist = s_hist[level];
        if (level > 0) {
          for (int t = wlo + lane; t - lane < whi; t += 32 * kEvUnroll) {
            uint32_t k[kEvUnroll];
            keys_at(t, k);
#pragma unroll
            for (int u = 0; u < kEvUnroll; ++u) {
              if (t - lane + 32 * u >= whi) break;
              tally(hist, k[u] != kKeyHeld && k[u] != kKeyOut && (k[u] >> (32 - width)) == prefix,
                    (k[u] >> shift) & ((1u << bits) - 1u));
            }
          }
          cluster.sync();
        }
        // bins from the top: thread i owns bins 2047 - 2 i and 2046 - 2 i
        const int b0 = kEvBins - 1 - 2 * tid, b1 = b0 - 1;
        int c0 = hist[b0], c1 = hist[b1];
        if (ncta > 1) {
          // CTA r adds up its share of the bins over the cluster, then every CTA
          // reads the sums: 2 + 2 remote reads a thread, not 2 per CTA
          const int share = kEvBins / ncta, part = kEvThreads / share;  // threads per bin (ncta / 2)
          const int bin = rank * share + tid % share;
          int sum = 0;
          for (int c = tid / share; c < ncta; c += part) sum += cluster.map_shared_rank(hist, c)[bin];
          if (tid < share) s_sum[tid] = 0;
          __syncthreads();
          if (part > 1) atomicAdd(&s_sum[tid % share], sum);
          else s_sum[tid] = sum;
          cluster.sync();
          c0 = cluster.map_shared_rank(s_sum, b0 / share)[b0 % share];
          c1 = cluster.map_shared_rank(s_sum, b1 / share)[b1 % share];
        }
        int v = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += u;
        }
        int total;
        const int before = warp_prefix(__shfl_sync(0xffffffffu, v, 31), s_warp, total) + v - (c0 + c1);
        if (before < need && before + c0 >= need) {
          s_bin = b0;
          s_above = before;
        } else if (before + c0 < need && before + c0 + c1 >= need) {
          s_bin = b1;
          s_above = before + c0;
        }
        __syncthreads();
        prefix = (prefix << bits) | static_cast<uint32_t>(s_bin);
        need -= s_above;
        width += bits;
        __syncthreads();
      }
      threshold = prefix;
      threshold_need = need;
    }
  }

  // ---- ranks.  A word per 32 rows: the rows above the threshold, and those at it
  const int words = (whi - wlo + 31) / 32;
  const size_t mask_words = (static_cast<size_t>(P.max_len) + 31) / 32;
  uint32_t* keep_w = P.cached ? s_keys + P.rows_per_cta + (wlo - lo) / 32
                              : P.masks + static_cast<size_t>(b) * 2 * mask_words + wlo / 32;
  uint32_t* equal_w = keep_w + (P.cached ? P.rows_per_cta / 32 : mask_words);
  // the lowest bits of the word of rows t0 .. t0 + 31 up to row `end`
  auto rows_below = [](int t0, int end) -> uint32_t {
    const int k = min(max(end - t0, 0), 32);
    return k == 32 ? 0xffffffffu : (1u << k) - 1u;
  };
  int hole = 0, move = 0;  // this lane's, then its warp's
  if (!all) {
    const bool ties = threshold_need > 0;
    int eq = 0;
    for (int t = wlo + lane, i = 0; i < words; t += 32 * kEvUnroll, i += kEvUnroll) {
      uint32_t k[kEvUnroll];
      keys_at(t, k);
#pragma unroll
      for (int u = 0; u < kEvUnroll; ++u) {
        const unsigned m = __ballot_sync(0xffffffffu, k[u] > threshold || (!ties && k[u] == threshold));
        const unsigned e = __ballot_sync(0xffffffffu, ties && k[u] == threshold);
        eq += __popc(e);
        if (lane == u && i + u < words) {
          keep_w[i + u] = m;
          equal_w[i + u] = e;
        }
      }
    }
    __syncwarp();
    int eq_before = 0;
    if (ties) {  // equal keys: the lower rows stay
      int total;
      eq_before = warp_prefix(eq, s_warp, total);
      if (tid == 0) s_cta[2] = total;
      cluster.sync();
      const int v = from_cluster(cluster, &s_cta[2], ncta, s_all[2]);
      eq_before += warp_sum(lane < rank ? v : 0);
    }
    for (int i0 = 0; i0 < words; i0 += 32) {
      const int i = i0 + lane, t0 = wlo + 32 * i;
      uint32_t keep = i < words ? keep_w[i] : 0u, e = i < words ? equal_w[i] : 0u;
      const int mine = __popc(e);
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += u;
      }
      const int sum = __shfl_sync(0xffffffffu, before, 31);
      int take = min(max(threshold_need - (eq_before + before - mine), 0), mine);
      if (take == mine) {
        keep |= e;
      } else {
        for (; take > 0; --take, e &= e - 1u) keep |= e & (0u - e);
      }
      eq_before += sum;
      if (i < words) keep_w[i] = keep;
      const uint32_t front = rows_below(t0, n);
      hole += __popc(rows_below(t0, whi) & front & ~keep);
      move += __popc(keep & ~front);
    }
    __syncwarp();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    hole += __shfl_xor_sync(0xffffffffu, hole, o);
    move += __shfl_xor_sync(0xffffffffu, move, o);
  }
  int hole_total, move_total;
  int hole_at = warp_prefix(hole, s_warp, hole_total);
  int move_at = warp_prefix(move, s_warp, move_total);
  if (tid == 0) {
    s_cta[3] = hole_total;
    s_cta2 = move_total;
  }
  cluster.sync();
  const int holes_of = from_cluster(cluster, &s_cta[3], ncta, s_all[3]), moves_of = from_cluster(cluster, &s_cta2, ncta, s_all[4]);
  const int moves = warp_sum(moves_of);
  hole_at += warp_sum(lane < rank ? holes_of : 0);
  move_at += warp_sum(lane < rank ? moves_of : 0);
  // ---- lists, and the rows that stay where they are
  const size_t row0 = static_cast<size_t>(b) * P.max_len;
  bool no_page = false;
  const bool copies = P.weights_out != P.weights || (P.order_out && P.order_out != P.order) || P.kept;
  const unsigned below = (1u << lane) - 1u;
  for (int i = 0; i < words; ++i) {
    const int t0 = wlo + 32 * i, t = t0 + lane;
    const uint32_t there = rows_below(t0, whi), front = rows_below(t0, n), keep = all ? there : keep_w[i];
    const uint32_t hm = there & front & ~keep, mm = keep & ~front;
    if (((hm | mm) >> lane) & 1u) {
      const int phys = physical_row(P, b, t);
      no_page |= phys < 0;
      if ((hm >> lane) & 1u)
        P.dst[static_cast<size_t>(b) * P.cap + hole_at + __popc(hm & below)] = make_int2(t, phys);
      else
        P.src[static_cast<size_t>(b) * P.cap + move_at + __popc(mm & below)] = make_int2(t, phys);
    }
    hole_at += __popc(hm);
    move_at += __popc(mm);
    if (copies && ((keep & front) >> lane) & 1u) {
      if (P.weights_out != P.weights) P.weights_out[row0 + t] = w[t];
      if (P.order_out && P.order_out != P.order) P.order_out[row0 + t] = age ? age[t] : t;
      if (P.kept) P.kept[static_cast<size_t>(b) * P.budget + t] = t;
    }
  }
  if (P.kept)
    for (int t = n + rank * kEvThreads + tid; t < P.budget; t += ncta * kEvThreads)
      P.kept[static_cast<size_t>(b) * P.budget + t] = -1;
  if (no_page) s_bad = 1;
  // every CTA has read seq_lens (new_lens may be the same array) and s_bad,
  // s_cta of its neighbours before any of them goes
  cluster.sync();
  if (rank == 0 && warp == 0) {
    const bool bad = lane < ncta && *cluster.map_shared_rank(&s_bad, lane);
    const bool any = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      if (b == 0) *P.status = 0u;
      P.flags[b] = bad_len || any ? kDevBounds : 0u;
      P.moves[b] = moves;
      P.new_lens[b] = n;
    }
  }
  cluster.sync();
}

// Bulk copies by one thread: shared -> global, and the waits for its stores to
// have been read out of shared memory, and to be complete.
__device__ __forceinline__ void bulk_store(void* dst, const void* src_smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src_smem)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A warp per moved row and turn: its cache rows go through the warp's slot of
// shared memory as bulk copies (no registers hold them, and up to 216 KB of an SM
// are under way), its per-row data by the lanes meanwhile.  A row longer than a
// slot goes in parts.  It lets no dependent start early: a decode launched next
// reads the cache at once, before it waits for the launch before it.
__global__ void __launch_bounds__(32 * kMoveWarps, 1) lrkv_evict_move_kernel(const EvictParams P) {
  extern __shared__ __align__(128) unsigned char s_rows[];  // [warps][slot]
  __shared__ uint64_t full[kMoveWarps];
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) {
    mbar_init(&full[warp], 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  asm volatile("fence.proxy.async.global;" ::: "memory");  // rows of earlier kernels' plain stores, read by bulk copies
  const int m = P.moves[b];
  long long at[5] = {0};  // where each tensor's part of a row begins, in bytes
#pragma unroll
  for (int s = 0; s < 4; ++s) at[s + 1] = at[s] + 16ll * P.n16[s];
  const size_t row0 = static_cast<size_t>(b) * P.max_len;
  const int2* src = P.src + static_cast<size_t>(b) * P.cap;
  const int2* dst = P.dst + static_cast<size_t>(b) * P.cap;
  unsigned char* slot = s_rows + static_cast<size_t>(warp) * P.slot;
  uint32_t phase = 0;
  // (the hardware suspends a waiting thread for longer than a row's copy takes: a
  // shorter bound is polled)
  auto landed = [&](uint32_t parity) {
    if (P.wait_limit >= kWaitLimitCycles) return mbar_wait_bounded(&full[warp], parity, P.wait_limit);
    const long long t0 = clock64();
    while (!mbar_test(&full[warp], parity))
      if (clock64() - t0 > P.wait_limit) return false;
    return true;
  };
  bool ok = true;
  const int stride = gridDim.x * warps;
  int k = blockIdx.x * warps + warp;
  int2 from = make_int2(-1, -1), to = from;
  if (k < m) {
    from = src[k];
    to = dst[k];
  }
  while (k < m && ok) {
    const int f = from.x, d = to.x;
    const bool paged_in = from.y >= 0 && to.y >= 0;
    const size_t fp = static_cast<size_t>(max(from.y, 0)), dp = static_cast<size_t>(max(to.y, 0));
    k += stride;
    bool rest = true;  // the per-row data and the next row's numbers are to do
    for (long long c0 = 0; c0 < at[4] && ok; c0 += P.slot) {
      const long long c1 = min(c0 + P.slot, at[4]);
      if (paged_in && lane == 0) {
        bulk_wait_read();
        mbar_arrive_expect_tx(&full[warp], static_cast<uint32_t>(c1 - c0));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const long long a = max(c0, at[s]), e = min(c1, at[s + 1]);
          if (a < e)
            tma_load_1d(slot + (a - c0), P.base[s] + fp * (at[s + 1] - at[s]) + (a - at[s]),
                        static_cast<uint32_t>(e - a), &full[warp]);
        }
      }
      if (rest) {
        rest = false;
        if (k < m) {
          from = src[k];
          to = dst[k];
        }
        if (P.key_scale)
          for (int h = lane; h < P.H; h += 32) {
            float* row = P.key_scale + (static_cast<size_t>(b) * P.H + h) * P.max_len;
            row[d] = row[f];
          }
        if (P.positions && lane < P.axes) P.positions[(row0 + d) * P.axes + lane] = P.positions[(row0 + f) * P.axes + lane];
        if (lane == 4) P.weights_out[row0 + d] = P.weights[row0 + f];
        if (lane == 5 && P.order_out) P.order_out[row0 + d] = P.order ? P.order[row0 + f] : f;
        if (lane == 6 && P.kept) P.kept[static_cast<size_t>(b) * P.budget + d] = f;
      }
      if (!paged_in) break;
      ok = landed(phase & 1u);
      ok = __all_sync(0xffffffffu, ok);
      ++phase;
      if (ok && lane == 0) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const long long a = max(c0, at[s]), e = min(c1, at[s + 1]);
          if (a < e)
            bulk_store(P.base[s] + dp * (at[s + 1] - at[s]) + (a - at[s]), slot + (a - c0), static_cast<uint32_t>(e - a));
        }
        bulk_commit();
      }
    }
  }
  if (lane == 0) {
    bulk_wait_all();
    if (!ok) {
      mbar_wait_bounded(&full[warp], (phase - 1u) & 1u);  // a late copy lands before the block ends
      atomicOr(P.status, kDevTimeout);
    }
  }
  if (blockIdx.x == 0 && b == 0 && warp == 0) {
    uint32_t bits = 0u;
    for (int i = lane; i < P.B; i += 32) bits |= P.flags[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
    if (lane == 0 && bits) atomicOr(P.status, bits);  // (the selection cleared it)
  }
}

// ======================================================================= host
namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

lrkv_status evict_check(int batch, int max_len, int budget) {
  if (batch < 1 || max_len < 1 || budget < 1 || budget > max_len) return LRKV_ERR_INVALID_ARG;
  // row numbers rounded up to a CTA's stay in 32 bits
  if (batch > kMaxBatch || static_cast<long long>(batch) * max_len > (1LL << 31) - (1 << 16)) return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

size_t evict_layout(EvictParams& P, void* ws) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  P.cap = std::min(P.budget, P.max_len - P.budget);
  const size_t list = up256(static_cast<size_t>(P.B) * P.cap * sizeof(int2));
  size_t off = 256;
  const size_t off_flags = off; off += up256(static_cast<size_t>(P.B) * 4);
  const size_t off_moves = off; off += up256(static_cast<size_t>(P.B) * 4);
  const size_t off_src = off; off += list;
  const size_t off_dst = off; off += list;
  const size_t off_masks = off; off += up256(static_cast<size_t>(P.B) * 2 * ((static_cast<size_t>(P.max_len) + 31) / 32) * 4);
  if (ws) {
    P.status = reinterpret_cast<uint32_t*>(base);
    P.flags = reinterpret_cast<uint32_t*>(base + off_flags);
    P.moves = reinterpret_cast<int32_t*>(base + off_moves);
    P.src = reinterpret_cast<int2*>(base + off_src);
    P.dst = reinterpret_cast<int2*>(base + off_dst);
    P.masks = reinterpret_cast<uint32_t*>(base + off_masks);
  }
  return off;
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shared memory of the selection for `rows` cached rows: a key and two bits each.
constexpr int select_smem(int rows) { return rows * 4 + rows / 16 * 4; }
constexpr int select_smem_max = select_smem(kEvCacheRows);

// Whether a cluster of kEvMaxCluster selection CTAs (more than the portable 8:
// the kernel's opt-in is set here) can run on the current device.
bool wide_clusters_fit(int smem) {
  static std::mutex mu;
  static std::map<int, bool> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lock(mu);
  const auto it = known.find(dev);
  if (it != known.end()) return it->second;
  const void* select = reinterpret_cast<const void*>(&lrkv_evict_select_kernel);
  int n = 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kEvMaxCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kEvMaxCluster);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool fits = ensure_kernel_smem(select, smem) == cudaSuccess &&
                    cudaFuncSetAttribute(select, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, select, &cfg) == cudaSuccess && n >= 1;
  known[dev] = fits;
  return fits;
}

}  // namespace

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_evict_workspace_size(int batch, int max_len, int budget, size_t* bytes) {
  if (!bytes) return LRKV_ERR_INVALID_ARG;
  const lrkv_status st = lrkv::evict_check(batch, max_len, budget);
  if (st != LRKV_OK) return st;
  lrkv::EvictParams P;
  std::memset(&P, 0, sizeof(P));
  P.B = batch; P.max_len = max_len; P.budget = budget;
  *bytes = lrkv::evict_layout(P, nullptr);
  return LRKV_OK;
}

lrkv_status lrkv_evict(const lrkv_dims* dims, int budget, int sink, int recent, const float* weights,
                       const int32_t* order, const int32_t* seq_lens, int page_size, int num_pages,
                       const int32_t* block_table, void* k_s, void* v_s, void* z_k, void* z_v, float* key_scale,
                       int32_t* positions, int axes, float* weights_out, int32_t* order_out, int32_t* new_lens,
                       int32_t* kept, void* ws, size_t ws_bytes, lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_evict");
  using namespace lrkv;
  if (!dims) return LRKV_ERR_INVALID_ARG;
  if (dims->heads < 1 || dims->head_dim < 1 || dims->rank < 0) return LRKV_ERR_INVALID_ARG;
  if (dims->dtype != LRKV_F32 && dims->dtype != LRKV_BF16) return LRKV_ERR_INVALID_ARG;
  lrkv_status st = evict_check(dims->batch, dims->max_len, budget);
  if (st != LRKV_OK) return st;
  if (sink < 0 || recent < 0 || static_cast<long long>(sink) + recent > budget) return LRKV_ERR_INVALID_ARG;
  if (!weights || !seq_lens || !k_s || !v_s || !weights_out || !new_lens) return LRKV_ERR_INVALID_ARG;
  if (dims->rank > 0 && (!z_k || !z_v)) return LRKV_ERR_INVALID_ARG;
  if (positions ? (axes < 1 || axes > 4) : axes != 0) return LRKV_ERR_INVALID_ARG;
  const int esz = dims->dtype == LRKV_BF16 ? 2 : 4;
  const long long shared = static_cast<long long>(dims->head_dim) * esz;
  const long long latent = static_cast<long long>(dims->heads) * dims->rank * esz;
  if (shared % 16 != 0 || latent % 16 != 0 || shared > (1 << 24) || latent > (1 << 24)) return LRKV_ERR_UNSUPPORTED;
  if (!a16(k_s) || !a16(v_s) || (dims->rank > 0 && (!a16(z_k) || !a16(z_v)))) return LRKV_ERR_INVALID_ARG;
  int shift = 0;
  if (block_table) {
    if (page_size < 1 || (page_size & (page_size - 1)) != 0 || num_pages < 1 || dims->max_len % page_size != 0)
      return LRKV_ERR_INVALID_ARG;
    if (static_cast<long long>(num_pages) * page_size > (1LL << 31) - 1) return LRKV_ERR_UNSUPPORTED;
    while ((1 << shift) < page_size) ++shift;
  }
  if (!ws) return LRKV_ERR_WORKSPACE;
  if (!a16(ws)) return LRKV_ERR_INVALID_ARG;
  EvictParams P;
  std::memset(&P, 0, sizeof(P));
  P.B = dims->batch; P.max_len = dims->max_len; P.budget = budget; P.sink = sink; P.recent = recent;
  if (ws_bytes < evict_layout(P, ws)) return LRKV_ERR_WORKSPACE;
  P.block_table = block_table;
  P.page_shift = shift;
  P.num_pages = num_pages;
  P.max_blocks = block_table ? dims->max_len / page_size : 0;
  P.seq_lens = seq_lens; P.weights = weights; P.order = order;
  P.weights_out = weights_out; P.order_out = order_out; P.new_lens = new_lens; P.kept = kept;
  P.n16[0] = P.n16[1] = static_cast<int>(shared / 16);
  P.n16[2] = P.n16[3] = static_cast<int>(latent / 16);
  P.base[0] = static_cast<unsigned char*>(k_s); P.base[1] = static_cast<unsigned char*>(v_s);
  P.base[2] = static_cast<unsigned char*>(z_k); P.base[3] = static_cast<unsigned char*>(z_v);
  P.H = dims->heads; P.axes = axes;
  P.key_scale = key_scale; P.positions = positions;
  P.wait_limit = wait_limit_cycles();
  const int sms = device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;

  // CTAs per sequence: more while the sequences leave SMs idle and a CTA has
  // more than 6144 rows.  8 x 16K rows (when the moves took 72 us of it): 99 us
  // with 2 CTAs each (8192 rows), 95 us with 4, 94 us with 8, 120 us with 16; 32 x
  // 4.3K rows: 22.0 us with one, 24 us with 2 or 4 (the cluster's exchanges cost
  // more than the passes).
  int ncta = 1;
  while (ncta < kEvMaxCluster && 2LL * ncta * P.B <= sms && P.max_len > 6144LL * ncta) ncta *= 2;
  // 16 CTAs need an SM group that holds them all: asked once per device
  if (ncta > 8 && !wide_clusters_fit(select_smem_max)) ncta = 8;
  const int step = 32 * kEvWarps;
  P.rows_per_cta = ((P.max_len + ncta - 1) / ncta + step - 1) / step * step;
  P.cached = P.rows_per_cta <= kEvCacheRows;
  const int smem = P.cached ? select_smem(P.rows_per_cta) : 0;
  const void* select = reinterpret_cast<const void*>(&lrkv_evict_select_kernel);
  // (the kernel's static tables count towards the 48 KB that need no attribute)
  if (ensure_kernel_smem(select, select_smem_max) != cudaSuccess) return LRKV_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ncta;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.B * ncta);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, lrkv_evict_select_kernel, P) != cudaSuccess) return LRKV_ERR_CUDA;
  // the move: as many warps as slots of a whole row fit, two CTAs per SM over all
  // sequences (one runs at a time, the second evens out the sequences)
  const long long row_bytes = 2 * (shared + latent);
  P.slot = static_cast<int>(std::min<long long>(kMoveSlotMax, (row_bytes + 127) / 128 * 128));
  const int warps = std::min(kMoveWarps, kMoveSmem / P.slot);
  if (ensure_kernel_smem(reinterpret_cast<const void*>(&lrkv_evict_move_kernel), kMoveSmem) != cudaSuccess)
    return LRKV_ERR_CUDA;
  const long long per_seq = std::max(1LL, (2LL * sms + P.B - 1) / P.B);
  const long long turns = (P.cap + warps - 1) / warps;
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(1LL, std::min(turns, per_seq))), P.B);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = warps * P.slot;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lrkv_evict_move_kernel, P) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

}  // extern "C"
