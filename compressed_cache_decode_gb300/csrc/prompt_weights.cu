// prompt_weights.cu — attention weights of a prompt's queries summed per cache
// row (lrkv_prefill_weights):
//
//   w'[j] = decay w[j] + sum over the last `window` queries i and the heads h
//           of [j <= pos(i)] exp(s_hij - lse_hi),
//   s_hij = scale (q_hi . k_s,j + (q_hi B_h^K) . z_k,hj) [key_scale_hj]
//
// with the log-sum-exp the prefill returned, so no softmax statistics are
// formed again and the values are not read.
//
// The sum runs over queries and heads, so the scores are formed transposed,
// S^T = K q^T, keys as the M rows of tcgen05.mma: a thread of the epilogue then
// owns one key (one TMEM lane), adds up its row in a register, and neither
// atomics nor exchanges between threads are needed.  p = q B_h^K enters as bf16
// high + low parts (lrkv_prefill_absorb_kernel), two MMAs over the same
// latents, as the prefill's own scores do: up to 2^-16 of |p| |z| off.  A third
// part, as the decode's weights take, is a query tile of 80 KB for 64, and the ring
// of two would leave no room for the keys' boxes.
//
// What bounds it: the rate at which one SM takes the MMAs.  For all the queries
// of 2 x 4K prompts (32 heads, d_h 128, rank 64: 108.6 us of tensor work at the
// rate of a large bf16 product, p's two parts counted) the call takes 260 us:
// 33 for p, 217 for the scores, an N = 128 instruction every 75 cycles of an SM
// (64 of tensor work) but for the 20% of the time that a half waits for its
// accumulator to be read back and the 8% for queries and k_s.  What was tried, at
// that shape:
//   - both operands in shared memory: an N = 128 instruction reads 8 KB for 64
//     cycles of work and took ~95.  So the keys, the same for every query of the
//     item (k_s) or of the head (z_k,h), are the A operand from TMEM: 548 -> 312 us.
//   - one issuing thread takes ~95 cycles an instruction: a thread per M half,
//     each with its accumulator and its ring of latents: 312 -> 253 us.
//   - a cluster of two sharing the query tiles by multicast (345 us) and query
//     copies of 32 KB in a deeper ring (350 us) were slower than one CTA's 312.
// An item is (sequence, 256 keys as two halves of 128 lanes, group of heads), so
// that a tile of queries (64 KB with its absorbed parts) is copied once for two
// halves: with one half the copies alone took longer than the MMAs.  A tile is
// `wt` queries of `hpt` heads, 128 columns at most: short windows put several
// heads side by side, whose shared part is one MMA.
//
// A window of one tile (ONE) uses each latent box once: it stays in shared memory
// as the A operand, and its TMEM takes a second k_s buffer, so the next item's
// keys are moved during this one.  4 x 16K keys of 32 heads, rank 64, window 32
// (277 MB, 41.5 us at the copy rate): 115 us with the boxes moved, 84 us so.  There
// the issuing threads wait for latents a fifth of the time and for k_s 8%; in the
// rest an SM takes an instruction (N = 32, one head) every 80 cycles, for 16 of
// tensor work and 40 of operand reads.  Four issuing threads, each with half of a
// tile's heads, took 106 us where two took 95.  For the long windows the
// boxes moved to TMEM are better: read from shared memory for each of a head's
// tiles, even with the TMEM they free as a third accumulator, 233 us for 217.
//
// Persistent: one CTA per SM walks the items, those with the most queries (the
// first keys) first and dealt in a snake; the rings run on across items.
// Warp 0 copies the keys' boxes (TMA), warp 2 the query tiles (and blanks the
// queries that give nothing: 1 us of the 84); warps 4-7 move
// keys to TMEM; one thread of warp 1 and one of warp 24 issue the MMAs of a half
// each; warp 3 lays down the log-sum-exps; warps 8-23 read the accumulators back.
// Each item leaves one partial sum per key; the last kernel adds the head groups'
// partials in order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "cache_weights.h"
#include "decode_common.cuh"
#include "decode_plan.h"
#include "host_cache.h"
#include "lrkv.h"
#include "ptx.cuh"
#include "tmap.h"
#include "trace.h"

namespace lrkv {

using namespace dec;

namespace {

constexpr int kPwThreads = 800;   // 25 warps (roles above)
constexpr int kPwEpi = 16;        // epilogue warps: four per lane quadrant, a 32-column chunk each
constexpr int kPwHalf = 128;      // keys of an M half (TMEM lanes)
constexpr int kPwKeys = 256;      // keys of an item
constexpr int kPwCols = 128;      // query columns of a tile
constexpr int kPwBox = 16384;     // one 128-row x 64-column operand box
constexpr int kPwA = 4;           // ring of key boxes in shared memory
constexpr int kPwQ = 2;           // ring of query tiles (64 KB: queries, absorbed high and low parts)
constexpr int kPwZ = 4;           // latent boxes in TMEM (32 columns each): a ring of two per M half
constexpr int kPwAcc = 2;         // accumulators (128 columns each)
constexpr int kPwL = 4;           // ring of log-sum-exp tiles in shared memory
constexpr int kColK = kPwAcc * kPwCols;         // TMEM: accumulators | k_s of two halves | latents
constexpr int kColZ = kColK + 128;
constexpr int kPwTmem = 512;
constexpr int kAbThreads = 128;   // absorb: four warps of 16 queries each

struct PromptParams {
  int B, H, dh, r, max_len, q_len, window;
  int wt, wt_log, hpt, nqt;  // queries (2^wt_log) and heads of a tile, tiles of the window
  int hg, nhg, nkt;          // heads of an item, head groups, key tiles
  int kr;                    // 16-wide steps over the latents
  int box_rows;              // rows of one key copy: 128, or the page size when smaller
  int page_shift, num_pages, max_blocks;
  long long items;
  float scale_log2;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const __nv_bfloat16* q;
  const __nv_bfloat16* b_k;
  const float* lse;          // [B][H][q_len]
  const float* key_scale;    // [B][H][max_len] or NULL
  __nv_bfloat16* p;          // [B][H][nqt wt][128]: 64 high parts, 64 low parts
  float* partial;            // [nhg][B][max_len]
  uint32_t* cta_status;      // [grid]
  int grid;
  long long wait_limit;      // bound of the roles' waits (SM cycles)
};

struct PromptMaps {
  CUtensorMap k;  // k_s rows: (d_h, rows, sequences or pages), box (64, box_rows, 1)
  CUtensorMap z;  // z_k: (r, H, rows, sequences or pages), box (64, 1, box_rows, 1)
  CUtensorMap q;  // q: (64, q_len, H, d_h / 64, B), box (64, wt, hpt, d_h / 64, 1)
  CUtensorMap p;  // p: (64, nqt wt, H, 2, B), box (64, wt, hpt, 2, 1)
};

// The items a CTA works through, in the same order for every role: round k takes
// item k G + c, or k G + G - 1 - c in odd rounds (items fall in work, so the
// CTAs' totals stay level).  An item's units: its heads hpt at a time, for each
// the query tiles qt0 .. nqt - 1.
struct Walk {
  int round;
  int b, h0, kt, L;     // sequence, first head of the group, key tile, length
  int halves;           // M halves that hold visible keys
  int qt0;              // first tile that sees the keys
  int n;                // items begun, minus one

  __device__ __forceinline__ bool open(const PromptParams& P) {
    const int G = gridDim.x, c = blockIdx.x;
    for (;; ++round) {
      const long long base = static_cast<long long>(round) * G;
      if (base >= P.items) return false;
      const long long item = base + ((round & 1) ? G - 1 - c : c);
      if (item >= P.items) continue;
      const int per = P.B * P.nhg;
      kt = static_cast<int>(item / per);
      const int rest = static_cast<int>(item % per);
      b = rest / P.nhg;
      h0 = (rest % P.nhg) * P.hg;
      L = min(max(P.seq_lens[b], P.q_len), P.max_len);
      if (kt * kPwKeys < L) break;
    }
    halves = kt * kPwKeys + kPwHalf < L ? 2 : 1;
    qt0 = max(0, kt * kPwKeys - (L - P.window)) / P.wt;
    ++n;
    return true;
  }
  __device__ __forceinline__ bool first(const PromptParams& P) {
    round = 0;
    n = -1;
    return open(P);
  }
  __device__ __forceinline__ bool next(const PromptParams& P) {
    ++round;
    return open(P);
  }
};

// Two fp32 values in one 64-bit register, for the two-wide fp32 instructions.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sum over a 32-column chunk of 2^(score s - lse), nlse holding -lse (log2
// domain, -inf where a column counts for nothing); with MASKED only the columns
// whose query index (column modulo wt) is at least t_min.  s0 scales the first
// 16 columns, s1 the others.
template <bool MASKED>
__device__ __forceinline__ float chunk_sum(const uint32_t (&v)[32], const float* nlse, float s0, float s1, int col,
                                           int wt, int t_min) {
  uint64_t sum[2] = {0ull, 0ull};
  const uint64_t sa = pair(s0, s0), sb = pair(s1, s1);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(nlse + e);
    const uint64_t s2 = e < 16 ? sa : sb;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = e + 2 * k;
      const uint64_t x = fma2(pair(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), s2, k ? l.y : l.x);
      float a, b;
      unpair(x, a, b);
      a = exp2_fast(a);
      b = exp2_fast(b);
      if (MASKED) {
        a = ((col + i) & (wt - 1)) < t_min ? 0.f : a;
        b = ((col + i + 1) & (wt - 1)) < t_min ? 0.f : b;
      }
      sum[k] = add2(sum[k], pair(a, b));
    }
  }
  float a, b, c, d;
  unpair(sum[0], a, b);
  unpair(sum[1], c, d);
  return (a + b) + (c + d);
}

}  // namespace

// p = q_h B_h^K of the window's queries in fp32 (mma.sync: exact bf16
// products), split into bf16 high and low parts; rows past the window and
// columns past the rank are zeros.  64 queries of one head per CTA; the query
// rows and B_h come in 16-byte pieces, and the two parts leave through shared
// memory as 256-byte rows.
__global__ void __launch_bounds__(kAbThreads) lrkv_prefill_absorb_kernel(const PromptParams P) {
  extern __shared__ __align__(16) unsigned char ab_raw[];
  const int rp = P.kr * 16, zs = rp + 8, qs = P.dh + 8;
  __nv_bfloat16* sB = reinterpret_cast<__nv_bfloat16*>(ab_raw);  // [dh][rp + 8]
  __nv_bfloat16* sQ = sB + P.dh * zs;                            // [64][dh + 8], then [64][128 + 8]
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * 64;
  const int wp = P.nqt * P.wt;
  const size_t tok = static_cast<size_t>(P.H) * P.dh;
  const __nv_bfloat16* qw = P.q + (static_cast<size_t>(b) * P.q_len + P.q_len - P.window) * tok +
                            static_cast<size_t>(h) * P.dh;
  const int pieces = P.dh / 8;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 8
  for (int i = tid; i < 64 * pieces; i += kAbThreads) {
    const int t = i / pieces, c = i % pieces;
    *reinterpret_cast<uint4*>(sQ + t * qs + 8 * c) =
        t0 + t < P.window ? *reinterpret_cast<const uint4*>(qw + (t0 + t) * tok + 8 * c) : zero;
  }
  const __nv_bfloat16* bh = P.b_k + static_cast<size_t>(h) * P.dh * P.r;
  if ((reinterpret_cast<uintptr_t>(P.b_k) & 15u) == 0) {
    const int pr = rp / 8;
#pragma unroll 8
    for (int i = tid; i < P.dh * pr; i += kAbThreads) {
      const int d = i / pr, c = i % pr;
      *reinterpret_cast<uint4*>(sB + d * zs + 8 * c) =
          8 * c < P.r ? *reinterpret_cast<const uint4*>(bh + static_cast<size_t>(d) * P.r + 8 * c) : zero;
    }
  } else {
    for (int i = tid; i < P.dh * rp; i += kAbThreads) {
      const int d = i / rp, c = i % rp;
      sB[d * zs + c] = c < P.r ? bh[static_cast<size_t>(d) * P.r + c] : __float2bfloat16_rn(0.f);
    }
  }
  __syncthreads();
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  for (int kk = 0; kk < P.dh / 16; ++kk) {
    uint32_t a0, a1, a2, a3;
    ldsm_x4(a0, a1, a2, a3, sQ + (16 * warp + (lane & 15)) * qs + 16 * kk + 8 * (lane >> 4));
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if (8 * j < rp) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_trans(b0, b1, b2, b3, sB + (16 * kk + (lane & 15)) * zs + 8 * j + 8 * (lane >> 4));
        mma_bf16_16816(acc[j], a0, a1, a2, a3, b0, b1);
        mma_bf16_16816(acc[j + 1], a0, a1, a2, a3, b2, b3);
      }
    }
  }
  __syncthreads();  // every warp has read its queries: their rows now take the results
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t = 16 * warp + g + 8 * u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = acc[j][2 * u], y = acc[j][2 * u + 1];
      const __nv_bfloat162 hi = __floats2bfloat162_rn(x, y);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(x - __low2float(hi), y - __high2float(hi));
      __nv_bfloat162* row = reinterpret_cast<__nv_bfloat162*>(sQ + t * 136 + 8 * j + 2 * q4);
      row[0] = hi;
      row[32] = lo;
    }
  }
  __syncthreads();
  __nv_bfloat16* out = P.p + ((static_cast<size_t>(b) * P.H + h) * wp + t0) * 128;
#pragma unroll 8
  for (int i = tid; i < 64 * 16; i += kAbThreads) {
    const int t = i >> 4, c = i & 15;
    if (t0 + t < wp)
      *reinterpret_cast<uint4*>(out + static_cast<size_t>(t) * 128 + 8 * c) =
          *reinterpret_cast<const uint4*>(sQ + t * 136 + 8 * c);
  }
}

template <int DH, bool ONE>
__global__ void __launch_bounds__(kPwThreads, 1)
    lrkv_prefill_weights_kernel(const __grid_constant__ PromptParams P, const __grid_constant__ PromptMaps maps) {
  constexpr int NB = DH / 64;  // 64-column boxes of a shared row
  constexpr int kStage = (NB + 2) * kPwBox;
  constexpr int KB = ONE ? 2 : 1;  // k_s buffers in TMEM
  extern __shared__ __align__(16) unsigned char pw_raw[];
  __shared__ uint64_t afull[kPwA], aempty[kPwA], qfull[kPwQ], qempty[kPwQ], kready[KB], kfree[KB], kfull, zready[kPwZ], zfree[kPwZ],
      accf[kPwAcc], acce[kPwAcc], lfull[kPwL], lempty[kPwL], qland, mdone[2];
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail, s_bad;
  __shared__ int s_use[kPwA], s_k, s_q[kPwQ], s_land;  // uses of the boxes and tiles begun
  __shared__ __align__(16) float s_lse[kPwL][kPwCols];  // read four columns at a time
  __shared__ float s_part[2][4][2][kPwHalf];
  unsigned char* smem = pw_raw + ((1024u - (smem_u32(pw_raw) & 1023u)) & 1023u);
  unsigned char* s_aring = smem;                          // [kPwA] boxes
  unsigned char* s_kbox = s_aring + kPwA * kPwBox;        // ONE: the k_s box on its way to TMEM
  unsigned char* s_qring = s_kbox + (ONE ? kPwBox : 0);   // [kPwQ] tiles
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* fail = &s_fail;

  if (tid == 0) {
    for (int i = 0; i < kPwA; ++i) { mbar_init(&afull[i], 1); mbar_init(&aempty[i], ONE ? 1 : 4); }
    for (int i = 0; i < kPwQ; ++i) { mbar_init(&qfull[i], 1); mbar_init(&qempty[i], 2); }
    for (int i = 0; i < kPwZ; ++i) { mbar_init(&zready[i], 4); mbar_init(&zfree[i], 1); }
    for (int i = 0; i < kPwAcc; ++i) { mbar_init(&accf[i], 1); mbar_init(&acce[i], kPwEpi); }
    for (int i = 0; i < kPwL; ++i) { mbar_init(&lfull[i], 1); mbar_init(&lempty[i], kPwEpi); }
    for (int i = 0; i < KB; ++i) { mbar_init(&kready[i], 4); mbar_init(&kfree[i], 2); }
    mbar_init(&kfull, 1);
    mbar_init(&qland, 1);
    mbar_init(&mdone[0], 1);
    mbar_init(&mdone[1], 1);
    for (int i = 0; i < kPwA; ++i) s_use[i] = 0;
    s_fail = s_bad = s_k = s_q[0] = s_q[1] = s_land = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, kPwTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int ncols = P.wt * P.hpt;
  pdl_trigger();
  pdl_wait();

  // one thread's copy of a key box of half m: k_s columns 64 c .. (c >= 0), or the
  // latents of head -1 - c
  auto copy_box = [&](const Walk& w, int m, int c, unsigned char* dst, uint64_t* full) {
    const int row = w.kt * kPwKeys + m * kPwHalf;
    const int boxes = (min(kPwHalf, w.L - row) + P.box_rows - 1) / P.box_rows;  // copies of the visible rows
    const uint32_t box_bytes = static_cast<uint32_t>(P.box_rows) * 128u;
    mbar_arrive_expect_tx(full, box_bytes * boxes);
    for (int k = 0; k < boxes; ++k, dst += box_bytes) {
      int seq = w.b, r0 = row + k * P.box_rows;  // tensor-map coordinates of the copy
      if (P.block_table) {
        seq = P.block_table[static_cast<size_t>(w.b) * P.max_blocks + (r0 >> P.page_shift)];
        r0 &= (1 << P.page_shift) - 1;
        if (seq < 0 || seq >= P.num_pages) {  // no page of the pool: the copy fills zeros
          s_bad = 1;
          seq = P.num_pages;
        }
      }
      if (c >= 0)
        tma_load_3d(dst, &maps.k, 64 * c, r0, seq, full);
      else
        tma_load_4d(dst, &maps.z, 0, -1 - c, r0, seq, full);
    }
  };

  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, P.wait_limit); };
  if (warp == 0) {
    if (ONE && lane == 0) {
      // ---- the heads' latents one after another, both halves of each --------------
      int zi[2] = {0, 0};
      bool live = true;
      Walk w;
      for (bool more = w.first(P); more && live && !*fail; more = w.next(P))
        for (int i = 0; P.r > 0 && i < P.hg && live; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m >= w.halves) break;
            const int s = m * (kPwA / 2) + zi[m] % (kPwA / 2), u = zi[m] / (kPwA / 2);  // slot, use of it
            live = live && (u < 1 || wait(&aempty[s], static_cast<uint32_t>(u - 1) & 1u));
            if (!live) {
              *fail = 1;
              break;
            }
            copy_box(w, m, -1 - (w.h0 + i), s_aring + s * kPwBox, &afull[s]);
            ++zi[m];
            s_use[s] = u + 1;
          }
    } else if (lane == 0) {
      // ---- key boxes: k_s of both halves per item, then the heads' latents --------
      int ai = 0;
      bool live = true;
      Walk w;
      for (bool more = w.first(P); more && live && !*fail; more = w.next(P)) {
        const int nk = w.halves * NB, nz = P.r > 0 ? w.halves * P.hg : 0;
        for (int i = 0; i < nk + nz; ++i) {
          const int s = ai % kPwA, u = ai / kPwA;  // slot, use of it
          // let go by its readers and, since readers that gave up let go too, landed: a
          // second copy must never join a phase that is still pending
          const uint32_t last = static_cast<uint32_t>(u - 1) & 1u;
          live = u < 1 || (wait(&aempty[s], last) && wait(&afull[s], last));
          if (!live) {
            *fail = 1;
            break;
          }
          const bool is_k = i < nk;
          copy_box(w, is_k ? i / NB : (i - nk) % w.halves, is_k ? i % NB : -1 - (w.h0 + (i - nk) / w.halves),
                   s_aring + s * kPwBox, &afull[s]);
          ++ai;
          s_use[s] = u + 1;
        }
      }
    }
  } else if (warp == 2) {
    // ---- query tiles.  A query with log-sum-exp -inf gives nothing and may hold
    // anything (padding): its rows of a tile become zeros before the MMAs read it, so
    // that its scores are numbers.  Such a tile's copy lands on a barrier of its own. ----
    Walk w;
    bool more = w.first(P);
    int hs = w.h0, qt = w.qt0;
    float next[kPwCols / 32];  // log-sum-exps of the tile (w, hs, qt), under way a tile ahead
    auto load_next = [&]() {
#pragma unroll
      for (int k = 0; k < kPwCols / 32; ++k) {
        const int col = lane + 32 * k, i = qt * P.wt + (col & (P.wt - 1)), h = hs + (col >> P.wt_log);
        next[k] = col < ncols && i < P.window
                      ? P.lse[(static_cast<size_t>(w.b) * P.H + h) * P.q_len + P.q_len - P.window + i]
                      : 0.f;
      }
    };
    if (more) load_next();
    int ql = 0;
    bool live = true;
    for (int qi = 0; more; ++qi) {
      const int s = qi % kPwQ, b = w.b, h0 = hs, t0 = qt * P.wt;
      unsigned blank[kPwCols / 32], any = 0u;
#pragma unroll
      for (int k = 0; k < kPwCols / 32; ++k) any |= blank[k] = __ballot_sync(0xffffffffu, next[k] == -INFINITY);
      if (++qt == P.nqt) {
        if ((hs += P.hpt) == w.h0 + P.hg) {
          more = w.next(P);
          hs = w.h0;
        }
        qt = w.qt0;
      }
      if (more) load_next();
      live = !*fail && (qi < kPwQ || wait(&qempty[s], static_cast<uint32_t>(qi / kPwQ - 1) & 1u));
      live = __all_sync(0xffffffffu, live);
      if (!live) {
        *fail = 1;
        break;
      }
      unsigned char* st = s_qring + s * kStage;
      if (lane == 0) {
        uint64_t* full = any ? &qland : &qfull[s];
        mbar_arrive_expect_tx(full, static_cast<uint32_t>(ncols) * 128u * (NB + (P.r > 0 ? 2 : 0)));
        tma_load_5d(st, &maps.q, 0, P.q_len - P.window + t0, h0, 0, b, full);
        if (P.r > 0) tma_load_5d(st + NB * kPwBox, &maps.p, 0, t0, h0, 0, b, full);
        if (any) s_land = ql + 1;
      }
      if (any) {
        live = wait(&qland, static_cast<uint32_t>(ql++) & 1u);
        live = __all_sync(0xffffffffu, live);
        if (!live) {
          *fail = 1;
          break;
        }
        const int box = lane >> 3;  // 8 lanes a row of a box: NB of the queries, two of the absorbed parts
        unsigned char* at =
            st + (lane & 7) * 16 + (box < NB ? box * ncols * 128 : NB * kPwBox + (box - NB) * ncols * 128);
#pragma unroll
        for (int k = 0; k < kPwCols / 32; ++k)
          for (unsigned bits = blank[k]; bits; bits &= bits - 1u)
            if (box < NB || (P.r > 0 && box < NB + 2))
              *reinterpret_cast<uint4*>(at + (32 * k + __ffs(bits) - 1) * 128) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&qfull[s]);
      }
      if (lane == 0) s_q[s] = qi / kPwQ + 1;
    }
  } else if (warp == 1 || warp == 24) {
    if (lane == 0) {
      // ---- MMAs of M half m into accumulator m: a thread each, since issuing an
      // instruction takes a thread ~95 cycles for 64 of tensor work ------------------
      const int m = warp == 24;
      const uint32_t id_all = idesc_bf16(128, ncols, 0, 0), id_head = idesc_bf16(128, P.wt, 0, 0);
      const uint64_t d0 = smem_desc(smem_u32(s_qring), 16, 1024, 2);  // address field: 16-byte units, low bits
      const uint32_t box = static_cast<uint32_t>(ncols) * 8u, head = static_cast<uint32_t>(P.wt) * 8u;
      const uint32_t acc = tmem + m * kPwCols;
      const uint64_t a0 = smem_desc(smem_u32(s_aring + m * (kPwA / 2) * kPwBox), 16, 1024, 2);
      int x = 0, qi = 0, zi = 0;
      bool ok = true;
      Walk w;
      for (bool more = w.first(P); more && ok && !*fail; more = w.next(P)) {
        ok = wait(&kready[w.n % KB], static_cast<uint32_t>(w.n / KB) & 1u);
        const uint32_t ka = tmem + kColK + (w.n % KB) * 128 + m * (NB * 32);
        const bool on = m < w.halves;
        for (int hs = 0; hs < P.hg && ok; hs += P.hpt) {
          for (int qt = w.qt0; qt < P.nqt && ok; ++qt, ++qi) {
            const int s = qi % kPwQ;
            ok = wait(&qfull[s], static_cast<uint32_t>(qi / kPwQ) & 1u) &&
                 (!on || x < 1 || wait(&acce[m], static_cast<uint32_t>(x - 1) & 1u));
            if (!ok) break;
            if (on) {
              tc_fence_after();
              const uint64_t qd = d0 + static_cast<uint32_t>(s * (kStage / 16));
#pragma unroll
              for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_ts(acc, ka + c * 32 + kk * 8, qd + c * box + kk * 2, id_all, c + kk > 0 ? 1u : 0u);
              uint64_t hd = qd + NB * (kPwBox / 16);
              for (int i = 0; P.r > 0 && i < P.hpt; ++i, hd += head) {
                const int z = zi + i;
                const uint32_t at = acc + i * P.wt;
                if (ONE) {
                  const int sl = z % (kPwA / 2), bar = m * (kPwA / 2) + sl;
                  ok = wait(&afull[bar], static_cast<uint32_t>(z / (kPwA / 2)) & 1u);
                  if (!ok) break;
                  const uint64_t ad = a0 + static_cast<uint32_t>(sl * (kPwBox / 16));
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    if (kk < P.kr) {
                      tc_mma_ss(at, ad + kk * 2, hd + kk * 2, id_head, 1u);
                      tc_mma_ss(at, ad + kk * 2, hd + box + kk * 2, id_head, 1u);
                    }
                  tc_commit(&aempty[bar]);
                } else {
                  const int sl = m * (kPwZ / 2) + z % (kPwZ / 2);
                  if (qt == w.qt0) {
                    ok = wait(&zready[sl], static_cast<uint32_t>(z / (kPwZ / 2)) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                  }
                  const uint32_t za = tmem + kColZ + sl * 32;
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    if (kk < P.kr) {
                      tc_mma_ts(at, za + kk * 8, hd + kk * 2, id_head, 1u);
                      tc_mma_ts(at, za + kk * 8, hd + box + kk * 2, id_head, 1u);
                    }
                  if (qt + 1 == P.nqt) tc_commit(&zfree[sl]);
                }
              }
              if (!ok) break;
              tc_commit(&accf[m]);
              ++x;
            }
            tc_commit(&qempty[s]);
          }
          if (on) zi += P.hpt;
        }
        if (ok) tc_commit(&kfree[w.n % KB]);
      }
      tc_commit(&mdone[m]);  // every MMA issued, also by a pass that gave up within a tile
      if (!ok) *fail = 1;
    }
  } else if (warp == 3) {
    // ---- minus the log2-domain log-sum-exp of a tile's columns; -inf where a
    // column holds no query of the window or its query saw nothing (weight 0) ----
    bool ok = true;
    int u = 0;
    Walk w;
    for (bool more = w.first(P); more && ok; more = w.next(P))
      for (int hs = w.h0; hs < w.h0 + P.hg && ok; hs += P.hpt)
        for (int qt = w.qt0; qt < P.nqt; ++qt, ++u) {
          const int s = u % kPwL;
          ok = ok && !*fail && (u < kPwL || wait(&lempty[s], static_cast<uint32_t>(u / kPwL - 1) & 1u));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            *fail = 1;
            break;
          }
#pragma unroll
          for (int k = 0; k < kPwCols / 32; ++k) {
            const int col = lane + 32 * k, i = qt * P.wt + (col & (P.wt - 1)), h = hs + (col >> P.wt_log);
            float v = -INFINITY;
            if (col < ncols && i < P.window) {
              v = P.lse[(static_cast<size_t>(w.b) * P.H + h) * P.q_len + P.q_len - P.window + i];
              v = v == -INFINITY ? v : -v * kLog2e;
            }
            s_lse[s][col] = v;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&lfull[s]);
        }
  } else if (warp < 8) {
    // ---- key boxes to TMEM: lane = row of the half, two columns per 32-bit word ----
    const int quad = warp & 3, row = 32 * quad + lane;
    int ai = 0, z0 = 0, z1 = 0;
    bool ok = true;
    auto to_tmem = [&](const unsigned char* src, uint32_t col) {
      src += row * 128;
      uint32_t v[32];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 u = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
        v[4 * c] = u.x; v[4 * c + 1] = u.y; v[4 * c + 2] = u.z; v[4 * c + 3] = u.w;
      }
      tmem_st32(tmem + (static_cast<uint32_t>(32 * quad) << 16) + col, v);
      tmem_wait_st();
      fence_proxy_async_smem();  // the reads above before the slot's next copy
      __syncwarp();
    };
    auto move = [&](uint32_t col) {
      const int s = ai % kPwA;
      ok = ok && !*fail && wait(&afull[s], static_cast<uint32_t>(ai / kPwA) & 1u);
      ok = __all_sync(0xffffffffu, ok);  // the warp moves together
      if (ok)
        to_tmem(s_aring + s * kPwBox, col);
      else
        *fail = 1;
      if (lane == 0) mbar_arrive_cta(&aempty[s]);
      ++ai;
    };
    Walk w;
    for (bool more = w.first(P); more; more = w.next(P)) {
      const int buf = w.n % KB;
      if (ONE) {
        for (int i = 0; i < w.halves * NB; ++i, ++ai) {
          // one box at a time, copied by the first of these warps once all four have
          // read the one before; the first is under way before its place in TMEM is free
          asm volatile("bar.sync 2, 128;" ::: "memory");
          if (warp == 4 && lane == 0 && ok && !*fail) {
            copy_box(w, i / NB, i % NB, s_kbox, &kfull);
            s_k = ai + 1;
          }
          if (i == 0) {
            ok = ok && (w.n < KB || wait(&kfree[buf], static_cast<uint32_t>(w.n / KB - 1) & 1u));
            tc_fence_after();
          }
          ok = ok && !*fail && wait(&kfull, static_cast<uint32_t>(ai) & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (ok)
            to_tmem(s_kbox, kColK + buf * 128 + i * 32);
          else
            *fail = 1;
        }
      } else {
        ok = ok && (w.n < KB || wait(&kfree[buf], static_cast<uint32_t>(w.n / KB - 1) & 1u));
        tc_fence_after();
        for (int i = 0; i < w.halves * NB; ++i) move(kColK + i * 32);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&kready[buf]);
      for (int i = 0; !ONE && P.r > 0 && i < w.halves * P.hg; ++i) {
        const int m = i % w.halves, z = m ? z1++ : z0++, sl = m * (kPwZ / 2) + z % (kPwZ / 2);
        ok = ok && (z < kPwZ / 2 || wait(&zfree[sl], static_cast<uint32_t>(z / (kPwZ / 2) - 1) & 1u));
        tc_fence_after();
        move(kColZ + sl * 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&zready[sl]);
      }
    }
  } else if (warp < 24) {
    // ---- epilogue: key (TMEM lane) 32 quad + lane of a half, columns 32 part ..
    // 32 part + 31 of the tile ---------------------------------------------------
    const int quad = warp & 3, part = (warp - 8) >> 2, key = 32 * quad + lane;
    const bool mine = 32 * part < ncols;
    float total[2] = {0.f, 0.f};
    int x[2] = {0, 0}, u = 0;
    bool ok = true;
    Walk w;
    for (bool more = w.first(P); more; more = w.next(P)) {
      total[0] = total[1] = 0.f;
      for (int hs = w.h0; hs < w.h0 + P.hg; hs += P.hpt)
        for (int qt = w.qt0; qt < P.nqt; ++qt, ++u) {
          const float* lse = s_lse[u % kPwL] + 32 * part;
          ok = ok && !*fail && wait(&lfull[u % kPwL], static_cast<uint32_t>(u / kPwL) & 1u);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m >= w.halves) break;
            const int row = w.kt * kPwKeys + m * kPwHalf + key;
            ok = ok && !*fail && wait(&accf[m], static_cast<uint32_t>(x[m]) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            uint32_t v[32];
            if (!ok) {
              *fail = 1;
            } else if (mine) {
              tc_fence_after();
              tmem_ld32(tmem + (static_cast<uint32_t>(32 * quad) << 16) + m * kPwCols + 32 * part, v);
              tmem_wait_ld();
              tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(&acce[m]);  // the accumulator is free
            ++x[m];
            if (ok && mine) {
              float s0 = P.scale_log2, s1 = P.scale_log2;
              if (P.key_scale && row < w.L) {  // (the chunk spans at most two heads: wt >= 16)
                const float* kp = P.key_scale + (static_cast<size_t>(w.b) * P.H + hs) * P.max_len + row;
                s0 *= kp[static_cast<size_t>((32 * part) >> P.wt_log) * P.max_len];
                s1 *= kp[static_cast<size_t>((32 * part + 16) >> P.wt_log) * P.max_len];
              }
              // query t of the tile sees this key when t >= t_min
              const int first = w.L - P.window + qt * P.wt;
              if (w.kt * kPwKeys + m * kPwHalf + kPwHalf - 1 > first)
                total[m] += chunk_sum<true>(v, lse, s0, s1, 32 * part, P.wt, row - first);
              else
                total[m] += chunk_sum<false>(v, lse, s0, s1, 0, 0, 0);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&lempty[u % kPwL]);
        }
      // the four column parts meet (the array of an item's parity is written again
      // two items later, past a barrier its readers passed too)
      float (*sp)[2][kPwHalf] = s_part[w.n & 1];
      sp[part][0][key] = total[0];
      sp[part][1][key] = total[1];
      asm volatile("bar.sync 1, 512;" ::: "memory");
      if (part < 2) {
        const int row = w.kt * kPwKeys + part * kPwHalf + key;  // part 0 finishes half 0, part 1 half 1
        const float sum = (sp[0][part][key] + sp[1][part][key]) + (sp[2][part][key] + sp[3][part][key]);
        if (row < w.L)
          P.partial[(static_cast<size_t>(w.h0 / P.hg) * P.B + w.b) * P.max_len + row] =
              ok ? sum : __int_as_float(0x7fc00000);
      }
    }
  }
  // every copy and MMA issued is complete before the block gives up its shared
  // memory and tensor memory
  __syncthreads();
  if (tid == 0) {
    bool done = true;
    for (int i = 0; i < kPwA; ++i)
      if (s_use[i] > 0) done = mbar_wait_bounded(&afull[i], static_cast<uint32_t>(s_use[i] - 1) & 1u) && done;
    if (s_k > 0) done = mbar_wait_bounded(&kfull, static_cast<uint32_t>(s_k - 1) & 1u) && done;
    for (int i = 0; i < kPwQ; ++i)
      if (s_q[i] > 0) done = mbar_wait_bounded(&qfull[i], static_cast<uint32_t>(s_q[i] - 1) & 1u) && done;
    if (s_land > 0) done = mbar_wait_bounded(&qland, static_cast<uint32_t>(s_land - 1) & 1u) && done;
    for (int i = 0; i < 2; ++i) done = mbar_wait_bounded(&mdone[i], 0u) && done;
    P.cta_status[blockIdx.x] = (s_fail || !done ? kDevTimeout : 0u) | (s_bad ? kDevBounds : 0u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kPwTmem);
}

// weights_out = decay * earlier weight (rows before the prompt's own) + the
// head groups' partials in order.
__global__ void __launch_bounds__(256)
    lrkv_prefill_weights_sum_kernel(const PromptParams P, float decay, const float* weights, float* weights_out,
                                    uint32_t* status) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, len = P.seq_lens[b];
  const int L = min(max(len, P.q_len), P.max_len);
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j < L) {
    float sum = 0.f;
    const size_t step = static_cast<size_t>(P.B) * P.max_len, at = static_cast<size_t>(b) * P.max_len + j;
#pragma unroll 4
    for (int g = 0; g < P.nhg; ++g) sum += P.partial[g * step + at];
    if (decay != 0.f && j < L - P.q_len) sum = fmaf(decay, weights[at], sum);
    weights_out[at] = sum;
  }
  if (blockIdx.x == 0 && b == 0 && threadIdx.x < 32) {
    uint32_t bits = 0u;
    for (int i = threadIdx.x; i < P.grid; i += 32) bits |= P.cta_status[i];
    for (int i = threadIdx.x; i < P.B; i += 32) {
      const int n = P.seq_lens[i];
      bits |= n < P.q_len || n > P.max_len ? kDevBounds : 0u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
    if (threadIdx.x == 0) *status = bits;
  }
}

// ======================================================================= host
namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

lrkv_status prompt_check(const lrkv_dims* d, int window) {
  if (!d || d->batch < 1 || d->heads < 1 || d->head_dim < 1 || d->rank < 0 || d->max_len < 1 || window < 1)
    return LRKV_ERR_INVALID_ARG;
  if (d->dtype != LRKV_F32 && d->dtype != LRKV_BF16) return LRKV_ERR_INVALID_ARG;
  if (!(d->scale == d->scale)) return LRKV_ERR_INVALID_ARG;
  if (d->dtype != LRKV_BF16 || (d->head_dim != 64 && d->head_dim != 128) || d->rank % 8 != 0 || d->rank > 64)
    return LRKV_ERR_UNSUPPORTED;
  if (d->batch > kMaxBatch || d->heads > 256 || window > d->max_len ||
      static_cast<long long>(d->batch) * d->max_len > (1LL << 31) - (1 << 16))  // rows rounded up stay in 32 bits
    return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

struct PromptLayout {
  size_t p, partial, status, bytes;
};

// Tile shape, item split and workspace (a status word, p, the partials, a word
// per CTA).
PromptLayout prompt_plan(const lrkv_dims& d, int window, int sms, PromptParams& P) {
  P.B = d.batch; P.H = d.heads; P.dh = d.head_dim; P.r = d.rank; P.max_len = d.max_len;
  P.window = window;
  // a tile: a power of two of queries (at least 16, at most 128) of as many
  // heads as fit 128 columns (a power of two dividing H), 32 columns at least
  P.wt = 16;
  while (P.wt < window && P.wt < kPwCols) P.wt *= 2;
  P.hpt = 1;
  while (2 * P.hpt * P.wt <= kPwCols && P.H % (2 * P.hpt) == 0) P.hpt *= 2;
  if (P.wt * P.hpt < 32) P.wt = 32;
  P.wt_log = 0;
  while ((1 << P.wt_log) < P.wt) ++P.wt_log;
  P.nqt = (window + P.wt - 1) / P.wt;
  P.kr = (P.r + 15) / 16;
  P.nkt = (P.max_len + kPwKeys - 1) / kPwKeys;
  // head groups: until there are three items per SM, or six when a window is one
  // tile, where the items are equal and the last round's idle SMs cost most (4 x
  // 16K keys of 32 heads: three 100 us, six 95)
  const long long want = (P.nqt == 1 ? 6LL : 3LL) * sms;
  P.hg = P.H;
  while (P.hg % (2 * P.hpt) == 0 && static_cast<long long>(P.nkt) * P.B * (P.H / P.hg) < want) P.hg /= 2;
  P.nhg = P.H / P.hg;
  P.items = static_cast<long long>(P.nkt) * P.B * P.nhg;
  P.grid = static_cast<int>(std::min<long long>(sms, P.items));
  PromptLayout l;
  l.p = 256;
  l.partial = l.p + up256(static_cast<size_t>(P.B) * P.H * P.nqt * P.wt * 128 * 2);
  l.status = l.partial + up256(static_cast<size_t>(P.nhg) * P.B * P.max_len * 4);
  l.bytes = l.status + up256(static_cast<size_t>(P.grid) * 4);
  return l;
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_prefill_weights_workspace_size(const lrkv_dims* dims, int window, size_t* bytes) {
  if (!bytes) return LRKV_ERR_INVALID_ARG;
  const lrkv_status st = lrkv::prompt_check(dims, window);
  if (st != LRKV_OK) return st;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  lrkv::PromptParams P;
  std::memset(&P, 0, sizeof(P));
  *bytes = lrkv::prompt_plan(*dims, window, sms, P).bytes;
  return LRKV_OK;
}

lrkv_status lrkv_prefill_weights(const lrkv_dims* dims, int q_len, int window, const void* q, int page_size,
                                 int num_pages, const int32_t* block_table, const void* k_s, const void* z_k,
                                 const void* b_k, const float* key_scale, const float* lse,
                                 const int32_t* seq_lens, float decay, const float* weights, float* weights_out,
                                 void* ws, size_t ws_bytes, lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_prefill_weights");
  using namespace lrkv;
  lrkv_status st = prompt_check(dims, window);
  if (st != LRKV_OK) return st;
  if (q_len < window) return LRKV_ERR_INVALID_ARG;
  if (q_len > dims->max_len) return LRKV_ERR_UNSUPPORTED;
  if (!q || !k_s || !lse || !seq_lens || (dims->rank > 0 && (!z_k || !b_k))) return LRKV_ERR_INVALID_ARG;
  if (!a16(q) || !a16(k_s) || (dims->rank > 0 && !a16(z_k))) return LRKV_ERR_INVALID_ARG;
  if ((st = weights_check(decay, weights, weights_out)) != LRKV_OK) return st;
  int shift = 0;
  if (block_table) {
    if (page_size < 16 || (page_size & (page_size - 1)) != 0 || num_pages < 1 || dims->max_len % page_size != 0)
      return LRKV_ERR_INVALID_ARG;
    if (static_cast<long long>(num_pages) * page_size > (1LL << 31) - 1) return LRKV_ERR_UNSUPPORTED;
    while ((1 << shift) < page_size) ++shift;
  }
  if (!ws) return LRKV_ERR_WORKSPACE;
  if (!a16(ws)) return LRKV_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  PromptParams P;
  std::memset(&P, 0, sizeof(P));
  const PromptLayout l = prompt_plan(*dims, window, sms, P);
  if (ws_bytes < l.bytes) return LRKV_ERR_WORKSPACE;
  unsigned char* base = static_cast<unsigned char*>(ws);
  P.q_len = q_len;
  P.p = reinterpret_cast<__nv_bfloat16*>(base + l.p);
  P.partial = reinterpret_cast<float*>(base + l.partial);
  P.cta_status = reinterpret_cast<uint32_t*>(base + l.status);
  P.wait_limit = wait_limit_cycles();
  P.scale_log2 = (dims->scale > 0.f ? dims->scale : 1.f / std::sqrt(static_cast<float>(P.dh))) * dec::kLog2e;
  P.block_table = block_table;
  P.page_shift = shift;
  P.num_pages = num_pages;
  P.max_blocks = block_table ? P.max_len / page_size : 0;
  P.box_rows = block_table ? std::min(page_size, kPwHalf) : kPwHalf;
  P.seq_lens = seq_lens; P.lse = lse; P.key_scale = key_scale;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.b_k = static_cast<const __nv_bfloat16*>(b_k);

  PromptMaps m;
  std::memset(&m, 0, sizeof(m));
  const uint64_t dh = P.dh, H = P.H, r = P.r, B = P.B, Q = q_len;
  const uint64_t rows = block_table ? page_size : P.max_len, seqs = block_table ? num_pages : P.B;
  const uint64_t wp = static_cast<uint64_t>(P.nqt) * P.wt;
  const uint32_t nb = P.dh / 64, wt = P.wt, hpt = P.hpt;
  const uint64_t qd[5] = {64, Q, H, nb, B}, qs[4] = {H * dh * 2, dh * 2, 128, Q * H * dh * 2};
  const uint32_t qb[5] = {64u, wt, hpt, nb, 1u}, pb[5] = {64u, wt, hpt, 2u, 1u};
  if (!make_tmap_3d_bf16(&m.k, k_s, dh, rows, seqs, 64u, P.box_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_5d_bf16_swizzled(&m.q, q, qd, qs, qb))
    return LRKV_ERR_CUDA;
  if (P.r > 0) {
    const uint64_t zd[4] = {r, H, rows, seqs}, zs[3] = {r * 2, H * r * 2, rows * H * r * 2};
    const uint32_t zb[4] = {64u, 1u, static_cast<uint32_t>(P.box_rows), 1u};
    const uint64_t pd[5] = {64, wp, H, 2, B}, ps[4] = {256, wp * 256, 128, H * wp * 256};
    if (!make_tmap_4d_bf16_swizzled(&m.z, z_k, zd, zs, zb) || !make_tmap_5d_bf16_swizzled(&m.p, P.p, pd, ps, pb))
      return LRKV_ERR_CUDA;
  }
  using Fn = void (*)(const PromptParams, const PromptMaps);
  const bool one = P.nqt == 1;
  const Fn kern = P.dh == 128 ? (one ? lrkv_prefill_weights_kernel<128, true> : lrkv_prefill_weights_kernel<128, false>)
                              : (one ? lrkv_prefill_weights_kernel<64, true> : lrkv_prefill_weights_kernel<64, false>);
  const int smem = 1024 + (kPwA + one + kPwQ * (P.dh / 64 + 2)) * kPwBox;
  if (ensure_kernel_smem(reinterpret_cast<const void*>(kern), smem, true) != cudaSuccess) return LRKV_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (P.r > 0) {
    const int ab_smem = (P.dh * (P.kr * 16 + 8) + 64 * 136) * 2;  // (d_h + 8 <= 136)
    lrkv_prefill_absorb_kernel<<<dim3(static_cast<unsigned>((wp + 63) / 64), P.H, P.B), kAbThreads, ab_smem, s>>>(P);
    if (cudaGetLastError() != cudaSuccess) return LRKV_ERR_CUDA;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.grid);
  cfg.blockDim = dim3(kPwThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, P, m) != cudaSuccess) return LRKV_ERR_CUDA;
  cfg.gridDim = dim3((P.max_len + 255) / 256, P.B);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, lrkv_prefill_weights_sum_kernel, P, decay, weights, weights_out,
                            static_cast<uint32_t*>(ws)) == cudaSuccess
             ? LRKV_OK
             : LRKV_ERR_CUDA;
}

}  // extern "C"
