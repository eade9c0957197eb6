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
// atomics nor exchanges between threads are needed.  CTA item = (sequence, 128
// keys, group of heads); k_s of the keys stays in shared memory for the item,
// z_k,h for the queries of a head; tiles of up to 128 query columns (`wt`
// queries of `hpt` heads: short windows put several heads side by side, whose
// shared part is one MMA) stream through a ring.  p = q B_h^K enters as bf16
// high + low parts (lrkv_prefill_absorb_kernel), two MMAs over the same
// latents, as the prefill's own scores do.
//
// Persistent: one CTA per SM walks the items, those with the most queries
// (the first keys) first; the rings run on across items.  Warp 0 copies (TMA),
// one thread of warp 1 issues the MMAs into four TMEM accumulators, warps 2-9
// read them back.  Each item leaves one partial sum per key; the last kernel
// adds the head groups' partials in order.
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

constexpr int kPwThreads = 320;   // copy warp, MMA warp, eight epilogue warps
constexpr int kPwKeys = 128;      // keys of an item (TMEM lanes)
constexpr int kPwCols = 128;      // query columns of a tile
constexpr int kPwSlot = 16384;    // one 128-row x 64-column operand box
constexpr int kPwZ = 3;           // ring of latent boxes
constexpr int kPwQ = 6;           // ring of query boxes
constexpr int kPwAcc = 4;         // TMEM accumulators
constexpr int kAbThreads = 128;   // absorb: four warps of 16 queries

struct PromptParams {
  int B, H, dh, r, max_len, q_len, window;
  int wt, hpt, nqt;          // queries and heads of a tile, tiles of the window
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
};

struct PromptMaps {
  CUtensorMap k;  // k_s rows: (d_h, rows, sequences or pages), box (64, box_rows, 1)
  CUtensorMap z;  // z_k: (r, H, rows, sequences or pages), box (64, 1, box_rows, 1)
  CUtensorMap q;  // q: (d_h, q_len, H, B), box (64, wt, hpt, 1)
  CUtensorMap p;  // p: (128, nqt wt, H, B), box (64, wt, hpt, 1)
};

// The units (query tiles) a CTA works through, in the same order for every
// role: items blockIdx.x, + gridDim.x, ..., in each its heads and their tiles.
struct Walk {
  long long item;
  int b, h0, kt, L;     // item: sequence, first head of the group, key tile, length
  int hs, qt, qt0;      // unit: first head, query tile; first tile that sees the keys
  int n;                // items begun, minus one
  bool new_item, new_head, last_of_item, last_of_head;

  __device__ __forceinline__ bool open(const PromptParams& P) {
    for (; item < P.items; item += gridDim.x) {
      const int per = P.B * P.nhg;
      kt = static_cast<int>(item / per);
      const int rest = static_cast<int>(item % per);
      b = rest / P.nhg;
      h0 = (rest % P.nhg) * P.hg;
      L = min(max(P.seq_lens[b], P.q_len), P.max_len);
      if (kt * kPwKeys < L) break;
    }
    if (item >= P.items) return false;
    qt0 = max(0, kt * kPwKeys - (L - P.window)) / P.wt;
    hs = h0;
    qt = qt0;
    ++n;
    new_item = new_head = true;
    marks(P);
    return true;
  }
  __device__ __forceinline__ void marks(const PromptParams& P) {
    last_of_head = qt + 1 == P.nqt;
    last_of_item = last_of_head && hs + P.hpt == h0 + P.hg;
  }
  __device__ __forceinline__ bool first(const PromptParams& P) {
    item = blockIdx.x;
    n = -1;
    return open(P);
  }
  __device__ __forceinline__ bool next(const PromptParams& P) {
    if (last_of_item) {
      item += gridDim.x;
      return open(P);
    }
    new_item = false;
    new_head = last_of_head;
    if (last_of_head) {
      hs += P.hpt;
      qt = qt0;
    } else {
      ++qt;
    }
    marks(P);
    return true;
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace

// p = q_h B_h^K of the window's queries in fp32 (mma.sync: exact bf16
// products), split into bf16 high and low parts; rows past the window and
// columns past the rank are zeros.
__global__ void __launch_bounds__(kAbThreads) lrkv_prefill_absorb_kernel(const PromptParams P) {
  extern __shared__ __align__(16) unsigned char ab_raw[];
  __nv_bfloat16* sB = reinterpret_cast<__nv_bfloat16*>(ab_raw);  // [dh][rp + 8]
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y, rp = P.kr * 16, zs = rp + 8;
  const int wp = P.nqt * P.wt;
  for (int i = tid; i < P.dh * rp; i += kAbThreads) {
    const int d = i / rp, c = i - d * rp;
    sB[d * zs + c] = c < P.r ? P.b_k[(static_cast<size_t>(h) * P.dh + d) * P.r + c] : __float2bfloat16_rn(0.f);
  }
  __syncthreads();
  const int t0 = blockIdx.x * 64 + warp * 16;
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  const int ta = t0 + g, tb = ta + 8;
  const size_t tok = static_cast<size_t>(P.H) * P.dh;
  const __nv_bfloat16* qw = P.q + (static_cast<size_t>(b) * P.q_len + P.q_len - P.window) * tok +
                            static_cast<size_t>(h) * P.dh;
  for (int kk = 0; kk < P.dh / 16; ++kk) {
    const int k = 16 * kk + 2 * q4;
    const uint32_t a0 = ta < P.window ? *reinterpret_cast<const uint32_t*>(qw + ta * tok + k) : 0u;
    const uint32_t a1 = tb < P.window ? *reinterpret_cast<const uint32_t*>(qw + tb * tok + k) : 0u;
    const uint32_t a2 = ta < P.window ? *reinterpret_cast<const uint32_t*>(qw + ta * tok + k + 8) : 0u;
    const uint32_t a3 = tb < P.window ? *reinterpret_cast<const uint32_t*>(qw + tb * tok + k + 8) : 0u;
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
  __nv_bfloat16* out = P.p + ((static_cast<size_t>(b) * P.H + h) * wp) * 128;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t = u ? tb : ta;
    if (t >= wp) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = acc[j][2 * u], y = acc[j][2 * u + 1];
      const __nv_bfloat162 hi = __floats2bfloat162_rn(x, y);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(x - __low2float(hi), y - __high2float(hi));
      __nv_bfloat162* row = reinterpret_cast<__nv_bfloat162*>(out + static_cast<size_t>(t) * 128 + 8 * j + 2 * q4);
      row[0] = hi;
      row[32] = lo;
    }
  }
}

template <int DH>
__global__ void __launch_bounds__(kPwThreads, 1)
    lrkv_prefill_weights_kernel(const __grid_constant__ PromptParams P, const __grid_constant__ PromptMaps maps) {
  constexpr int NB = DH / 64;  // 64-column boxes of a shared row
  extern __shared__ __align__(16) unsigned char pw_raw[];
  __shared__ uint64_t kfull[2], kempty[2], zfull[kPwZ], zempty[kPwZ], qfull[kPwQ], qempty[kPwQ], accf[kPwAcc],
      acce[kPwAcc];
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail, s_bad;
  __shared__ int s_k, s_z, s_q, s_acc;  // boxes issued into each ring, units committed
  __shared__ __align__(16) float s_lse[2][kPwCols];  // read four columns at a time
  __shared__ float s_part[2][kPwKeys];
  unsigned char* smem = pw_raw + ((1024u - (smem_u32(pw_raw) & 1023u)) & 1023u);
  unsigned char* s_keys = smem;                              // [2][NB] boxes
  unsigned char* s_zring = s_keys + 2 * NB * kPwSlot;        // [kPwZ] boxes
  unsigned char* s_qring = s_zring + kPwZ * kPwSlot;         // [kPwQ] boxes
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* fail = &s_fail;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) { mbar_init(&kfull[i], 1); mbar_init(&kempty[i], 1); }
    for (int i = 0; i < kPwZ; ++i) { mbar_init(&zfull[i], 1); mbar_init(&zempty[i], 1); }
    for (int i = 0; i < kPwQ; ++i) { mbar_init(&qfull[i], 1); mbar_init(&qempty[i], 1); }
    for (int i = 0; i < kPwAcc; ++i) { mbar_init(&accf[i], 1); mbar_init(&acce[i], 8); }
    s_fail = s_bad = s_k = s_z = s_q = s_acc = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, kPwAcc * kPwCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int ncols = P.wt * P.hpt;
  pdl_trigger();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      // ---- copies ------------------------------------------------------------
      int zi = 0, qi = 0;
      Walk w;
      for (bool more = w.first(P); more && !*fail; more = w.next(P)) {
        const int row = w.kt * kPwKeys;
        const int boxes = (min(kPwKeys, w.L - row) + P.box_rows - 1) / P.box_rows;  // copies of the visible rows
        auto at = [&](int i, int& seq, int& r0) {  // tensor-map coordinates of copy i
          const int t = row + i * P.box_rows;
          if (!P.block_table) {
            seq = w.b;
            r0 = t;
          } else {
            seq = P.block_table[static_cast<size_t>(w.b) * P.max_blocks + (t >> P.page_shift)];
            r0 = t & ((1 << P.page_shift) - 1);
            if (seq < 0 || seq >= P.num_pages) {  // no page of the pool: the copy fills zeros
              s_bad = 1;
              seq = P.num_pages;
            }
          }
        };
        const uint32_t box_bytes = static_cast<uint32_t>(P.box_rows) * 128u;
        if (w.new_item) {
          const int kb = w.n & 1;
          if (w.n >= 2 && !mbar_wait_bounded(&kempty[kb], static_cast<uint32_t>(w.n / 2 - 1) & 1u)) {
            *fail = 1;
            break;
          }
          mbar_arrive_expect_tx(&kfull[kb], box_bytes * boxes * NB);
          for (int i = 0; i < boxes; ++i) {
            int seq, r0;
            at(i, seq, r0);
            for (int c = 0; c < NB; ++c)
              tma_load_3d(s_keys + (kb * NB + c) * kPwSlot + i * box_bytes, &maps.k, 64 * c, r0, seq, &kfull[kb]);
          }
          s_k = w.n + 1;
        }
        // the tile's queries, then their absorbed parts, then the latents
        bool live = true;
        for (int c = 0; c < NB + (P.r > 0 ? 2 : 0) && live; ++c) {
          const int s = qi % kPwQ;
          if (qi >= kPwQ && !mbar_wait_bounded(&qempty[s], static_cast<uint32_t>(qi / kPwQ - 1) & 1u)) {
            live = false;
            break;
          }
          mbar_arrive_expect_tx(&qfull[s], static_cast<uint32_t>(ncols) * 128u);
          if (c < NB)
            tma_load_4d(s_qring + s * kPwSlot, &maps.q, 64 * c, P.q_len - P.window + w.qt * P.wt, w.hs, w.b,
                        &qfull[s]);
          else
            tma_load_4d(s_qring + s * kPwSlot, &maps.p, 64 * (c - NB), w.qt * P.wt, w.hs, w.b, &qfull[s]);
          s_q = ++qi;
        }
        for (int i = 0; P.r > 0 && w.new_head && i < P.hpt && live; ++i) {
          const int s = zi % kPwZ;
          if (zi >= kPwZ && !mbar_wait_bounded(&zempty[s], static_cast<uint32_t>(zi / kPwZ - 1) & 1u)) {
            live = false;
            break;
          }
          mbar_arrive_expect_tx(&zfull[s], box_bytes * boxes);
          for (int j = 0; j < boxes; ++j) {
            int seq, r0;
            at(j, seq, r0);
            tma_load_4d(s_zring + s * kPwSlot + j * box_bytes, &maps.z, 0, w.hs + i, r0, seq, &zfull[s]);
          }
          s_z = ++zi;
        }
        if (!live) {
          *fail = 1;
          break;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMAs: unit u into accumulator u % kPwAcc ------------------------------
      const uint32_t id_all = idesc_bf16(128, ncols, 0, 0), id_head = idesc_bf16(128, P.wt, 0, 0);
      int u = 0, zi = 0, qi = 0;
      Walk w;
      for (bool more = w.first(P); more && !*fail; more = w.next(P), ++u) {
        const int kb = w.n & 1;
        const uint32_t acc = tmem + (u % kPwAcc) * kPwCols;
        bool ok = u < kPwAcc || mbar_wait_bounded(&acce[u % kPwAcc], static_cast<uint32_t>(u / kPwAcc - 1) & 1u);
        if (ok && w.new_item) ok = mbar_wait_bounded(&kfull[kb], static_cast<uint32_t>(w.n / 2) & 1u);
        for (int c = 0; c < NB && ok; ++c, ++qi) {
          const int s = qi % kPwQ;
          ok = mbar_wait_bounded(&qfull[s], static_cast<uint32_t>(qi / kPwQ) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ka = smem_u32(s_keys + (kb * NB + c) * kPwSlot), qa = smem_u32(s_qring + s * kPwSlot);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_ss(acc, smem_desc(ka + kk * 32, 16, 1024, 2), smem_desc(qa + kk * 32, 16, 1024, 2), id_all,
                      c + kk > 0 ? 1u : 0u);
          tc_commit(&qempty[s]);
        }
        if (ok && P.r > 0) {
          const int s0 = qi % kPwQ, s1 = (qi + 1) % kPwQ;
          ok = mbar_wait_bounded(&qfull[s0], static_cast<uint32_t>(qi / kPwQ) & 1u) &&
               mbar_wait_bounded(&qfull[s1], static_cast<uint32_t>((qi + 1) / kPwQ) & 1u);
          const uint32_t hi = smem_u32(s_qring + s0 * kPwSlot), lo = smem_u32(s_qring + s1 * kPwSlot);
          for (int i = 0; i < P.hpt && ok; ++i) {
            const int s = (zi + i) % kPwZ;
            if (w.new_head) ok = mbar_wait_bounded(&zfull[s], static_cast<uint32_t>((zi + i) / kPwZ) & 1u);
            if (!ok) break;
            tc_fence_after();
            const uint32_t za = smem_u32(s_zring + s * kPwSlot), off = i * P.wt * 128;
            for (int kk = 0; kk < P.kr; ++kk) {
              const uint64_t zd = smem_desc(za + kk * 32, 16, 1024, 2);
              tc_mma_ss(acc + i * P.wt, zd, smem_desc(hi + off + kk * 32, 16, 1024, 2), id_head, 1u);
              tc_mma_ss(acc + i * P.wt, zd, smem_desc(lo + off + kk * 32, 16, 1024, 2), id_head, 1u);
            }
            if (w.last_of_head) tc_commit(&zempty[s]);
          }
          if (ok) {
            tc_commit(&qempty[s0]);
            tc_commit(&qempty[s1]);
            qi += 2;
            if (w.last_of_head) zi += P.hpt;
          }
        }
        if (!ok) {
          *fail = 1;
          break;
        }
        if (w.last_of_item) tc_commit(&kempty[kb]);
        tc_commit(&accf[u % kPwAcc]);
        s_acc = u + 1;
      }
    }
  } else {
    // ---- epilogue: key (TMEM lane) 32 quad + lane; 32-column chunks of parity
    // `half` of the tile --------------------------------------------------------
    const int quad = warp & 3, half = (warp - 2) >> 2, key = 32 * quad + lane, et = tid - 64;
    // log2-domain log-sum-exp of column et of a unit; +inf where the column
    // holds no query of the window or its query saw nothing (weight 0)
    auto lse_of = [&](const Walk& w) {
      if (et >= ncols) return INFINITY;
      const int i = w.qt * P.wt + (et & (P.wt - 1)), h = w.hs + et / P.wt;
      if (i >= P.window) return INFINITY;
      const float v = P.lse[(static_cast<size_t>(w.b) * P.H + h) * P.q_len + P.q_len - P.window + i];
      return v == -INFINITY ? INFINITY : v * kLog2e;
    };
    Walk w;
    bool more = w.first(P), ok = true;
    if (more && et < kPwCols) s_lse[0][et] = lse_of(w);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float total = 0.f;
    for (int u = 0; more; ++u) {
      Walk nx = w;
      const bool more_next = nx.next(P);
      float lse_next = 0.f;
      if (more_next && et < kPwCols) lse_next = lse_of(nx);
      if (w.new_item) total = 0.f;
      const int row = w.kt * kPwKeys + key;
      if (ok && *fail) ok = false;
      if (ok) {
        ok = mbar_wait_bounded(&accf[u % kPwAcc], static_cast<uint32_t>(u / kPwAcc) & 1u);
        if (!ok) *fail = 1;
      }
      if (ok) {
        tc_fence_after();
        // query t of the tile sees this key when t >= t_min
        const int t_min = row - (w.L - P.window) - w.qt * P.wt;
        const bool masked = w.kt * kPwKeys + kPwKeys - 1 > w.L - P.window + w.qt * P.wt;
        const float* lse = s_lse[u & 1];
        for (int c = half; 32 * c < ncols; c += 2) {
          float sc = P.scale_log2;
          uint32_t v[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(32 * quad) << 16) + (u % kPwAcc) * kPwCols + 32 * c, v);
          float ks[2] = {1.f, 1.f};
          if (P.key_scale && row < w.L) {  // (a chunk spans at most two heads: wt >= 16)
            const size_t at = (static_cast<size_t>(w.b) * P.H + w.hs + 32 * c / P.wt) * P.max_len + row;
            ks[0] = ks[1] = P.key_scale[at];
            if (P.wt == 16) ks[1] = P.key_scale[at + P.max_len];
          }
          tmem_wait_ld();
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse + 32 * c + e);
            const float s2 = sc * ks[e >> 4];
            float x[4] = {exp2_fast(fmaf(__uint_as_float(v[e]), s2, -l4.x)),
                          exp2_fast(fmaf(__uint_as_float(v[e + 1]), s2, -l4.y)),
                          exp2_fast(fmaf(__uint_as_float(v[e + 2]), s2, -l4.z)),
                          exp2_fast(fmaf(__uint_as_float(v[e + 3]), s2, -l4.w))};
            if (masked) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (((32 * c + e + k) & (P.wt - 1)) < t_min) x[k] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[k] += x[k];
          }
          total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&acce[u % kPwAcc]);
      // (written again two items later, past a barrier its reader passed too)
      if (w.last_of_item && half == 1) s_part[w.n & 1][key] = total;
      if (more_next && et < kPwCols) s_lse[(u + 1) & 1][et] = lse_next;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (w.last_of_item && half == 0 && row < w.L)
        P.partial[(static_cast<size_t>(w.h0 / P.hg) * P.B + w.b) * P.max_len + row] =
            ok ? total + s_part[w.n & 1][key] : __int_as_float(0x7fc00000);
      w = nx;
      more = more_next;
    }
  }
  // every copy and MMA issued is complete before the block gives up its shared
  // memory and tensor memory
  __syncthreads();
  if (tid == 0) {
    bool done = true;
    for (int i = max(0, s_k - 2); i < s_k; ++i)
      done = mbar_wait_bounded(&kfull[i & 1], static_cast<uint32_t>(i / 2) & 1u) && done;
    for (int i = max(0, s_z - kPwZ); i < s_z; ++i)
      done = mbar_wait_bounded(&zfull[i % kPwZ], static_cast<uint32_t>(i / kPwZ) & 1u) && done;
    for (int i = max(0, s_q - kPwQ); i < s_q; ++i)
      done = mbar_wait_bounded(&qfull[i % kPwQ], static_cast<uint32_t>(i / kPwQ) & 1u) && done;
    for (int i = max(0, s_acc - kPwAcc); i < s_acc; ++i)
      done = mbar_wait_bounded(&accf[i % kPwAcc], static_cast<uint32_t>(i / kPwAcc) & 1u) && done;
    P.cta_status[blockIdx.x] = (s_fail || !done ? kDevTimeout : 0u) | (s_bad ? kDevBounds : 0u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kPwAcc * kPwCols);
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
      static_cast<long long>(d->batch) * d->max_len > (1LL << 31) - 1)
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
  P.nqt = (window + P.wt - 1) / P.wt;
  P.kr = (P.r + 15) / 16;
  P.nkt = (P.max_len + kPwKeys - 1) / kPwKeys;
  // head groups: until there are four items per SM
  P.hg = P.H;
  while (P.hg % (2 * P.hpt) == 0 && static_cast<long long>(P.nkt) * P.B * (P.H / P.hg) < 4LL * sms) P.hg /= 2;
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
  P.scale_log2 = (dims->scale > 0.f ? dims->scale : 1.f / std::sqrt(static_cast<float>(P.dh))) * dec::kLog2e;
  P.block_table = block_table;
  P.page_shift = shift;
  P.num_pages = num_pages;
  P.max_blocks = block_table ? P.max_len / page_size : 0;
  P.box_rows = block_table ? std::min(page_size, kPwKeys) : kPwKeys;
  P.seq_lens = seq_lens; P.lse = lse; P.key_scale = key_scale;
  P.q = static_cast<const __nv_bfloat16*>(q);
  P.b_k = static_cast<const __nv_bfloat16*>(b_k);

  PromptMaps m;
  std::memset(&m, 0, sizeof(m));
  const uint64_t dh = P.dh, H = P.H, r = P.r, B = P.B, Q = q_len;
  const uint64_t rows = block_table ? page_size : P.max_len, seqs = block_table ? num_pages : P.B;
  const uint64_t wp = static_cast<uint64_t>(P.nqt) * P.wt;
  const uint64_t qd[4] = {dh, Q, H, B}, qs[3] = {H * dh * 2, dh * 2, Q * H * dh * 2};
  const uint32_t qb[4] = {64u, static_cast<uint32_t>(P.wt), static_cast<uint32_t>(P.hpt), 1u};
  if (!make_tmap_3d_bf16(&m.k, k_s, dh, rows, seqs, 64u, P.box_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_4d_bf16_swizzled(&m.q, q, qd, qs, qb))
    return LRKV_ERR_CUDA;
  if (P.r > 0) {
    const uint64_t zd[4] = {r, H, rows, seqs}, zs[3] = {r * 2, H * r * 2, rows * H * r * 2};
    const uint32_t zb[4] = {64u, 1u, static_cast<uint32_t>(P.box_rows), 1u};
    const uint64_t pd[4] = {128, wp, H, B}, ps[3] = {256, wp * 256, H * wp * 256};
    if (!make_tmap_4d_bf16_swizzled(&m.z, z_k, zd, zs, zb) || !make_tmap_4d_bf16_swizzled(&m.p, P.p, pd, ps, qb))
      return LRKV_ERR_CUDA;
  }
  using Fn = void (*)(const PromptParams, const PromptMaps);
  const Fn kern = P.dh == 128 ? lrkv_prefill_weights_kernel<128> : lrkv_prefill_weights_kernel<64>;
  const int smem = 1024 + (2 * (P.dh / 64) + kPwZ + kPwQ) * kPwSlot;
  if (ensure_kernel_smem(reinterpret_cast<const void*>(kern), smem, true) != cudaSuccess) return LRKV_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (P.r > 0) {
    const int ab_smem = P.dh * (P.kr * 16 + 8) * 2;
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
