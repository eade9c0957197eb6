// decode_rope_axes.cu — decode with rotary positions that every cache row
// carries itself, on one or several axes (lrkv_decode_rope_axes): row j of
// sequence b sits at position positions[b][j][axis] on each axis, so rows may
// have been moved or evicted, and image and video tokens have their time,
// height and width.
//
// As in decode_rope.cu the rotation cannot be moved into the rank-r latent, so
// each key is rebuilt, k = s_j + z_j B_h^T, turned and dotted with the rotated
// query, and one online softmax per head runs over the rows; the values are
// not rotated.  Pair k turns by positions[axis(k)] theta_k: its (cos, sin) is
// entry k of the table's row of that position, so a row's rotation is gathered
// from up to `axes` table rows.
//
// Grid (range CTAs, groups of 8 heads), one warp per head (B_h's MMA fragments
// live in its registers), 16-token tiles of k_s, v_s and the group's z_k, z_v
// in a ring of TMA stages.  Per tile and warp: K = Z_h B_h^T on the tensor
// cores (mma.sync, fp32 accumulation), plus the shared row, dotted with the
// query turned back by the row's angles,
//   q~ . (k D) = x0 (qa cos + qb sin) + x1 (qb cos - qa sin)   per pair,
// three two-wide fp32 instructions; the values O^T += V^T p with the
// probabilities as a bf16 high part in one column of the B operand and the low
// part in the next, so that one MMA takes both.  The 16 rows' cos and sin are
// gathered by the whole CTA into one of two shared buffers: the table entries
// of tile j + 2 and the positions of tile j + 3 are loaded while tile j is
// computed, since the two dependent loads' latency in every tile took most of
// the time at first (4 x 32K rows, 32 heads: 950 us).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "decode_common.cuh"
#include "decode_plan.h"
#include "host_cache.h"
#include "cache_weights.h"
#include "lrkv.h"
#include "trace.h"
#include "ptx.cuh"
#include "rope_axes.h"
#include "tmap.h"

namespace lrkv {

using namespace dec;

namespace {

constexpr int kRT = 16;                      // tokens per tile
constexpr int kRHeads = 8;                   // heads per CTA, one consumer warp each
constexpr int kRThreads = 32 * kRHeads;
constexpr int kRHeader = 1024;               // barriers and stage records
constexpr int kRMaxStages = 16;
constexpr float kRRescaleLog2 = 8.f;         // raise the reference max only past 2^8

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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct AxesArgs {
  RopeAxes ax;
  const int32_t* positions;  // [B][max_len][axes]
};

}  // namespace

template <int DH, int R>
__global__ void __launch_bounds__(kRThreads, 1)
    lrkv_decode_rope_axes_kernel(const __grid_constant__ DecodePlan P, const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_zk,
                                 const __grid_constant__ CUtensorMap tm_zv, const __grid_constant__ AxesArgs A) {
  constexpr int NT = DH / 8;    // 8-column tiles of the rebuilt key
  constexpr int KS = R / 16;    // 16-wide steps over a head's latents
  constexpr int MV = DH / 16;   // 16-row tiles of the shared values
  constexpr int MZ = R / 16;    // 16-row tiles of the private values
  constexpr int NP = DH / 32;   // pairs a thread gathers per tile (one token, 16 threads)
  constexpr int CSR = DH + 8;   // floats per gathered row (rows 8 banks apart: no conflicts)
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ int s_timeout, s_badpos;
  __shared__ __align__(16) float s_cs[2][kRT * CSR];            // (cos, sin) per pair of the tile's rows
  __shared__ __align__(16) float4 s_q[kRHeads][DH / 2];         // (qa, qb, qb, -qa) per pair
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);

  pdl_trigger();  // the merge may launch: it waits for this grid before it reads
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const int B = P.B, H = P.H;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  int* issued = reinterpret_cast<int*>(smem + 256);  // [16] last tile issued into each stage
  int* pre = reinterpret_cast<int*>(smem + kRHeader);

  // ---- 1. barriers, sequence starts (clamped lengths) ----------------------
  if (tid == 0) {
    s_timeout = 0;
    s_badpos = 0;
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&full[s], 1);
      issued[s] = -1;
    }
    fence_barrier_init();
  }
  int bad = 0;
  for (int b = tid; b < B; b += blockDim.x) {
    int L = P.seq_lens[b];
    if (L < 0 || L > P.max_len) {
      bad = 1;
      L = min(max(L, 0), P.max_len);
    }
    pre[b + 1] = L;
  }
  if (tid == 0) pre[0] = 0;
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    int carry = 0;
    for (int base = 1; base <= B; base += 32) {
      const int i = base + lane;
      int v = (i <= B) ? pre[i] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (i <= B) pre[i] = v + carry;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  const int N = pre[B];
  const int G = max(1, min(static_cast<int>(gridDim.x), (N + P.min_tokens - 1) / max(P.min_tokens, 1)));
  uint32_t* cta_status = P.cta_status + blockIdx.y * gridDim.x + blockIdx.x;
  if (N == 0 || static_cast<int>(blockIdx.x) >= G) {
    pdl_wait();  // the launch before may still read the workspace
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      for (int b = tid; b <= B; b += blockDim.x) P.prefix[b] = pre[b];
      if (tid == 0) { P.meta[0] = N; P.meta[1] = G; }
    }
    if (tid == 0) *cta_status = bad ? kDevBounds : 0u;
    return;
  }
  const int c = blockIdx.x;
  const int g0 = static_cast<int>(static_cast<long long>(c) * N / G);
  const int g1 = static_cast<int>(static_cast<long long>(c + 1) * N / G);
  const int segrow = P.segp * 2;  // bytes per latent segment row

  const int zseg0 = blockIdx.y * P.nsb;
  const uint32_t tx = static_cast<uint32_t>(2 * (DH / 64) * kRT * 128 + 2 * P.zt_bytes);
  // the copies of tile j (sequence b, rows t0 ..) into its stage (one thread)
  auto issue = [&](int j, const TileWalk& t) {
    const int s = j % P.stages;
    unsigned char* ks = smem + P.off_kv + static_cast<size_t>(s) * P.stage_bytes;
    unsigned char* vs = ks + P.kv_bytes;
    unsigned char* zk = vs + P.kv_bytes;
    unsigned char* zv = zk + P.zt_bytes;
    mbar_arrive_expect_tx(&full[s], tx);
#pragma unroll
    for (int cb = 0; cb < DH / 64; ++cb) {
      tma_load_3d(ks + cb * kRT * 128, &tm_k, cb * 64, t.t0, t.b, &full[s]);
      tma_load_3d(vs + cb * kRT * 128, &tm_v, cb * 64, t.t0, t.b, &full[s]);
    }
    tma_load_4d(zk, &tm_zk, 0, t.t0, zseg0, t.b, &full[s]);
    tma_load_4d(zv, &tm_zv, 0, t.t0, zseg0, t.b, &full[s]);
    *reinterpret_cast<volatile int*>(&issued[s]) = j;
  };
  // the walk `stages` tiles ahead: the first stages' tiles go out now
  TileWalk ahead;
  bool ahead_more = walk_first(ahead, pre, B, g0, g1);
  for (int j = 0; j < P.stages && ahead_more; ++j) {
    if (tid == 0) issue(j, ahead);
    ahead_more = walk_next(ahead, pre, B, g1, kRT);
  }

  // ---- 2. the gather's roles: token tid / 16 of a tile, pairs NP (tid % 16) ..
  const int gt = tid >> 4, gk = NP * (tid & 15);
  int gaxis[NP];
#pragma unroll
  for (int u = 0; u < NP; ++u) gaxis[u] = A.ax.axis(gk + u);
  auto positions_of = [&](const TileWalk& t, int (&pos)[NP]) {
    const bool there = t.t0 + gt < t.t_end;
    const int32_t* row = A.positions + (static_cast<size_t>(t.b) * P.max_len + t.t0 + gt) * A.ax.n;
#pragma unroll
    for (int u = 0; u < NP; ++u) pos[u] = there ? __ldg(row + gaxis[u]) : 0;
  };
  auto entries_of = [&](const int (&pos)[NP], float2 (&cs)[NP]) {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int p = min(max(pos[u], 0), P.rope_max_pos - 1);
      if (p != pos[u]) *reinterpret_cast<volatile int*>(&s_badpos) = 1;
      cs[u] = __ldg(reinterpret_cast<const float2*>(P.rope_cs + static_cast<size_t>(p) * DH + 2 * (gk + u)));
    }
  };
  auto put = [&](int buf, const float2 (&cs)[NP]) {
#pragma unroll
    for (int u = 0; u < NP; u += 2)
      *reinterpret_cast<float4*>(&s_cs[buf][gt * CSR + 2 * (gk + u)]) =
          make_float4(cs[u].x, cs[u].y, cs[u + 1].x, cs[u + 1].y);
  };

  // ---- 3. this warp's head ------------------------------------------------------
  const int h = blockIdx.y * kRHeads + warp;
  // B_h^K as the B operand of K = Z_h B_h^T (k = latent column, n = head
  // dim): lane (g, q4) holds B_h[8 n + g][16 kk + 2 q4 (+1)] and [.. + 8 (+9)]
  uint32_t bf[NT][KS][2];
  {
    const __nv_bfloat16* bk = static_cast<const __nv_bfloat16*>(P.b_k) + static_cast<size_t>(h) * DH * R;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        const __nv_bfloat16* row = bk + (8 * n + g) * R + 16 * kk + 2 * q4;
        bf[n][kk][0] = *reinterpret_cast<const uint32_t*>(row);
        bf[n][kk][1] = *reinterpret_cast<const uint32_t*>(row + 8);
      }
  }
  const int zoff = (warp / P.hs) * (kRT * segrow) + (warp % P.hs) * R * 2;  // this head in a latent tile
  const int trow = (lane & 7) + 8 * (lane >> 4), tcol = (lane >> 3) & 1;    // transposed A operand (values)

  // tiles j (w), j + 2 (table entries) and j + 3 (positions)
  TileWalk w, wt;
  bool more = walk_first(w, pre, B, g0, g1);
  float2 cs[NP];
  int pos[NP];
  int known = 0;  // tiles seen ahead: cs holds tile 1's entries, pos tile 2's positions
  {
    wt = w;
    positions_of(wt, pos);
    entries_of(pos, cs);
    put(0, cs);
    if (walk_next(wt, pre, B, g1, kRT)) {
      known = 1;
      positions_of(wt, pos);
      entries_of(pos, cs);
      if (walk_next(wt, pre, B, g1, kRT)) {
        known = 2;
        positions_of(wt, pos);
      }
    }
  }
  bool ok = true, waited = false;
  int cur_b = -1;
  float m = -INFINITY, l = 0.f;
  // O_s^T and O_z^T: rows as in the accumulator layout, column 0 (lanes q4 = 0)
  // the high parts' sum, column 1 the low parts'
  float os[MV][4], oz[MZ][4];

  // this head's partial of sequence b: (m, l) and the unnormalised
  // [O_s | O_z] at slot b + c (the merge takes every CTA's)
  auto write_partial = [&](int b) {
    if (!waited) {
      pdl_wait();  // the launch before may still read the workspace
      waited = true;
    }
    const size_t slot = static_cast<size_t>(b + c);
    if (lane == 0) {
      float* pml = P.part_ml + (slot * H + h) * 2;
      pml[0] = m;
      pml[1] = l;
    }
    float* o = P.part_acc + (slot * H + h) * (DH + R);
    if (q4 == 0) {
#pragma unroll
      for (int e = 0; e < MV; ++e) {
        o[16 * e + g] = os[e][0] + os[e][1];
        o[16 * e + g + 8] = os[e][2] + os[e][3];
      }
#pragma unroll
      for (int e = 0; e < MZ; ++e) {
        o[DH + 16 * e + g] = oz[e][0] + oz[e][1];
        o[DH + 16 * e + g + 8] = oz[e][2] + oz[e][3];
      }
    }
  };

  __syncthreads();  // the first tile's rotations
  for (int j = 0; more; ++j) {
    // rotations ahead: tile j + 1's into the other buffer, j + 2's entries, j + 3's positions
    if (known >= 1) put((j + 1) & 1, cs);
    if (known >= 2) {
      entries_of(pos, cs);
      known = walk_next(wt, pre, B, g1, kRT) ? 2 : 1;
      if (known == 2) positions_of(wt, pos);
    } else {
      known = 0;
    }
    if (w.b != cur_b) {
      if (cur_b >= 0) write_partial(cur_b);
      cur_b = w.b;
      m = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int e = 0; e < MV; ++e) os[e][0] = os[e][1] = os[e][2] = os[e][3] = 0.f;
#pragma unroll
      for (int e = 0; e < MZ; ++e) oz[e][0] = oz[e][1] = oz[e][2] = oz[e][3] = 0.f;
      const __nv_bfloat16* qh = static_cast<const __nv_bfloat16*>(P.q) + (static_cast<size_t>(w.b) * H + h) * DH;
      __syncwarp();
      for (int k = lane; k < DH / 2; k += 32) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(qh + 2 * k);
        s_q[warp][k] = make_float4(bf_lo(v), bf_hi(v), bf_hi(v), -bf_lo(v));
      }
      __syncwarp();
    }
    const int s = j % P.stages;
    const int nvalid = min(kRT, w.t_end - w.t0);
    ok = ok && !*reinterpret_cast<volatile int*>(&s_timeout) &&
         mbar_wait_bounded(&full[s], static_cast<uint32_t>(j / P.stages) & 1u, P.wait_limit);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      *reinterpret_cast<volatile int*>(&s_timeout) = 1;
    } else {
      const unsigned char* ks = smem + P.off_kv + static_cast<size_t>(s) * P.stage_bytes;
      const unsigned char* vs = ks + P.kv_bytes;
      const unsigned char* zk = vs + P.kv_bytes;
      const unsigned char* zv = zk + P.zt_bytes;
      // ---- rebuilt key . turned query: tokens g and g + 8 ----
      uint32_t a[KS][4];
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
        ldsm_x4(a[kk][0], a[kk][1], a[kk][2], a[kk][3],
                zk + zoff + (lane & 15) * segrow + (16 * kk + 8 * (lane >> 4)) * 2);
      const float* cs0 = &s_cs[j & 1][g * CSR + 2 * q4];
      const float* cs1 = cs0 + 8 * CSR;
      const ulonglong2* qp = reinterpret_cast<const ulonglong2*>(&s_q[warp][q4]);
      uint64_t part0 = 0ull, part1 = 0ull;  // even and odd coordinates' sums
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += 4) {
        float acc[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u][0] = acc[u][1] = acc[u][2] = acc[u][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            mma_bf16_16816(acc[u], a[kk][0], a[kk][1], a[kk][2], a[kk][3], bf[n0 + u][kk][0], bf[n0 + u][kk][1]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int n = n0 + u, d = 8 * n + 2 * q4;
          const unsigned char* kb = ks + (d >> 6) * (kRT * 128);
          const uint32_t s0 = *reinterpret_cast<const uint32_t*>(kb + swz_off(g, (d & 63) >> 3, 128) + 4 * q4);
          const uint32_t s1 = *reinterpret_cast<const uint32_t*>(kb + swz_off(g + 8, (d & 63) >> 3, 128) + 4 * q4);
          const float2 c0 = *reinterpret_cast<const float2*>(cs0 + 8 * n);  // (cos, sin) of pair d / 2
          const float2 c1 = *reinterpret_cast<const float2*>(cs1 + 8 * n);
          const ulonglong2 qv = qp[4 * n];  // (qa, qb), (qb, -qa)
          const uint64_t x = add2(pair(acc[u][0], acc[u][1]), pair(bf_lo(s0), bf_hi(s0)));
          const uint64_t y = add2(pair(acc[u][2], acc[u][3]), pair(bf_lo(s1), bf_hi(s1)));
          part0 = fma2(x, fma2(pair(c0.x, c0.x), qv.x, mul2(pair(c0.y, c0.y), qv.y)), part0);
          part1 = fma2(y, fma2(pair(c1.x, c1.x), qv.x, mul2(pair(c1.y, c1.y), qv.y)), part1);
        }
      }
      float e0, e1, f0, f1;
      unpair(part0, e0, f0);
      unpair(part1, e1, f1);
      e0 += f0;
      e1 += f1;
      e0 += __shfl_xor_sync(0xffffffffu, e0, 1);
      e1 += __shfl_xor_sync(0xffffffffu, e1, 1);
      e0 += __shfl_xor_sync(0xffffffffu, e0, 2);
      e1 += __shfl_xor_sync(0xffffffffu, e1, 2);
      // ---- one online softmax over the tile (log2 domain) ----
      const float sc0 = g < nvalid ? e0 * P.scale_log2 : -INFINITY;
      const float sc1 = g + 8 < nvalid ? e1 * P.scale_log2 : -INFINITY;
      if (P.scores && q4 == 0) {
        if (!waited) {
          pdl_wait();  // the launch before may still read the workspace
          waited = true;
        }
        float* srow = P.scores + (static_cast<size_t>(w.b) * H + h) * P.max_len + w.t0;
        if (g < nvalid) srow[g] = sc0;
        if (g + 8 < nvalid) srow[g + 8] = sc1;
      }
      float mx = fmaxf(sc0, sc1);
#pragma unroll
      for (int o2 = 4; o2 < 32; o2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
      if (mx > m + kRRescaleLog2) {  // (the same for every lane)
        const float alpha = m == -INFINITY ? 0.f : exp2f(m - mx);
        m = mx;
        l *= alpha;
#pragma unroll
        for (int e = 0; e < MV; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) os[e][k] *= alpha;
#pragma unroll
        for (int e = 0; e < MZ; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) oz[e][k] *= alpha;
      }
      const float p0 = exp2f(sc0 - m), p1 = exp2f(sc1 - m);
      l += p0 + p1;  // this lane's tokens; the lanes meet at the end of the piece
      // P as the B operand: column 0 the bf16 high parts, column 1 the low parts
      // (lanes g = 0 and 1 hold tokens 2 q4, 2 q4 + 1 and + 8)
      uint32_t b0, b1;
      {
        const float ta = __shfl_sync(0xffffffffu, p0, 8 * q4), tb = __shfl_sync(0xffffffffu, p0, 8 * q4 + 4);
        const float tc = __shfl_sync(0xffffffffu, p1, 8 * q4), td = __shfl_sync(0xffffffffu, p1, 8 * q4 + 4);
        const uint32_t hi0 = pack_bf16(ta, tb), hi1 = pack_bf16(tc, td);
        const uint32_t lo0 = pack_bf16(ta - bf_lo(hi0), tb - bf_hi(hi0));
        const uint32_t lo1 = pack_bf16(tc - bf_lo(hi1), td - bf_hi(hi1));
        b0 = g == 0 ? hi0 : g == 1 ? lo0 : 0u;
        b1 = g == 0 ? hi1 : g == 1 ? lo1 : 0u;
      }
      // ---- values, unrotated: rows past the piece (which may hold anything)
      // must not meet their zero probabilities as 0 x NaN ----
      const uint32_t k0 = (2 * q4 < nvalid ? 0x0000ffffu : 0u) | (2 * q4 + 1 < nvalid ? 0xffff0000u : 0u);
      const uint32_t k1 = (2 * q4 + 8 < nvalid ? 0x0000ffffu : 0u) | (2 * q4 + 9 < nvalid ? 0xffff0000u : 0u);
#pragma unroll
      for (int e = 0; e < MV; ++e) {
        uint32_t v0, v1, v2, v3;
        const int ch = 2 * e + tcol;  // 16-byte chunk along the head dim
        ldsm_x4_trans(v0, v1, v2, v3, vs + (ch >> 3) * (kRT * 128) + swz_off(trow, ch & 7, 128));
        mma_bf16_16816(os[e], v0 & k0, v1 & k0, v2 & k1, v3 & k1, b0, b1);
      }
#pragma unroll
      for (int e = 0; e < MZ; ++e) {
        uint32_t v0, v1, v2, v3;
        ldsm_x4_trans(v0, v1, v2, v3, zv + zoff + trow * segrow + (16 * e + 8 * tcol) * 2);
        mma_bf16_16816(oz[e], v0 & k0, v1 & k0, v2 & k1, v3 & k1, b0, b1);
      }
    }
    more = walk_next(w, pre, B, g1, kRT);
    if (!more || w.b != cur_b) {  // the piece ends here: the lanes' denominators meet (each token on four lanes)
#pragma unroll
      for (int o2 = 4; o2 < 32; o2 <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
    }
    // the tile's readers are done (its stage is refilled with the tile `stages`
    // ahead) and the next tile's rotations are in place
    fence_proxy_async_smem();
    __syncthreads();
    if (ahead_more) {
      if (tid == 0 && !*reinterpret_cast<volatile int*>(&s_timeout)) issue(j + P.stages, ahead);
      ahead_more = walk_next(ahead, pre, B, g1, kRT);
    }
  }
  if (cur_b >= 0) write_partial(cur_b);

  // ---- every copy this CTA issued has landed before it exits ----
  __syncthreads();
  if (tid == 0) {
    pdl_wait();
    bool drained = true;
    for (int st = 0; st < P.stages; ++st) {
      const int j = *reinterpret_cast<volatile int*>(&issued[st]);
      if (j >= 0) drained = mbar_wait_bounded(&full[st], static_cast<uint32_t>(j / P.stages) & 1u) && drained;
    }
    if (!drained) *reinterpret_cast<volatile int*>(&s_timeout) = 1;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      P.meta[0] = N;
      P.meta[1] = G;
    }
    *cta_status = (bad || *reinterpret_cast<volatile int*>(&s_badpos) ? kDevBounds : 0u) |
                  (*reinterpret_cast<volatile int*>(&s_timeout) ? kDevTimeout : 0u);
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    pdl_wait();
    for (int b = tid; b <= B; b += blockDim.x) P.prefix[b] = pre[b];
  }
}

// ======================================================================= host
namespace {

using RopeFn = void (*)(const DecodePlan, const CUtensorMap, const CUtensorMap, const CUtensorMap,
                        const CUtensorMap, const AxesArgs);

template <int DH>
RopeFn rope_fn_r(int r) {
  switch (r) {
    case 16: return lrkv_decode_rope_axes_kernel<DH, 16>;
    case 32: return lrkv_decode_rope_axes_kernel<DH, 32>;
    case 48: return lrkv_decode_rope_axes_kernel<DH, 48>;
    case 64: return lrkv_decode_rope_axes_kernel<DH, 64>;
    default: return nullptr;
  }
}

RopeFn rope_fn(int dh, int r) {
  if (dh == 64) return rope_fn_r<64>(r);
  if (dh == 128) return rope_fn_r<128>(r);
  return nullptr;
}

lrkv_status rope_axes_check(const lrkv_dims* d) {
  if (!d) return LRKV_ERR_INVALID_ARG;
  if (d->batch < 1 || d->heads < 1 || d->head_dim < 1 || d->rank < 0 || d->max_len < 1) return LRKV_ERR_INVALID_ARG;
  if (d->dtype != LRKV_BF16 && d->dtype != LRKV_F32) return LRKV_ERR_INVALID_ARG;
  if (!(d->scale == d->scale)) return LRKV_ERR_INVALID_ARG;
  if (d->dtype != LRKV_BF16 || !rope_fn(d->head_dim, d->rank) || d->heads % kRHeads != 0) return LRKV_ERR_UNSUPPORTED;
  if (d->batch > kMaxBatch || static_cast<long long>(d->batch) * d->max_len > (1LL << 31) - 1)
    return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

lrkv_status rope_axes_plan(const lrkv_dims& d, int num_sms, DecodePlan& P, size_t* score_off, size_t* ws_bytes) {
  std::memset(&P, 0, sizeof(P));
  P.B = d.batch; P.H = d.heads; P.dh = d.head_dim; P.r = d.rank; P.max_len = d.max_len;
  P.map_len = d.max_len; P.map_seqs = d.batch;
  const float scale = d.scale > 0.f ? d.scale : 1.f / std::sqrt(static_cast<float>(d.head_dim));
  P.scale_log2 = scale * kLog2e;
  P.bf16 = 1; P.esz = 2; P.T = kRT; P.stream = 1;
  {
    const char* v = std::getenv("LRKV_WAIT_LIMIT_CYCLES");
    const long long x = (v && *v) ? std::atoll(v) : 0;
    P.wait_limit = x > 0 ? x : kWaitLimitCycles;
  }
  P.mt = P.H / kRHeads;
  P.grid = std::max(1, num_sms / P.mt);
  P.ngw = 1;
  P.hs = 0;
  for (int hs = kRHeads; hs >= 1; hs >>= 1)
    if (P.H % hs == 0 && (hs * P.r) % 16 == 0 && hs * P.r + 8 <= 256) { P.hs = hs; break; }
  if (P.hs == 0) return LRKV_ERR_UNSUPPORTED;
  P.segw = P.hs * P.r;
  P.segp = P.segw + 8;
  P.nsb = kRHeads / P.hs;
  P.zt_bytes = P.nsb * kRT * P.segp * 2;
  P.kv_bytes = round_up(kRT * P.dh * 2, 1024);
  P.stage_bytes = round_up(2 * P.kv_bytes + 2 * P.zt_bytes, 1024);
  P.off_prefix = kRHeader;
  P.off_kv = round_up(kRHeader + (P.B + 1) * 4, 1024);
  // less the static tables: two tiles of rotations, the queries
  const int budget = 226 * 1024 - 2 * kRT * (P.dh + 8) * 4 - kRHeads * (P.dh / 2) * 16;
  P.stages = std::min(kRMaxStages, (budget - P.off_kv - 1024) / P.stage_bytes);
  if (P.stages < 2) return LRKV_ERR_UNSUPPORTED;
  P.smem_bytes = P.off_kv + P.stages * P.stage_bytes + 1024;
  P.min_tokens = 8 * kRT;
  P.wide_merge = 1;
  P.wide_warps = 8;
  P.combine_ctas = static_cast<int>(std::min<long long>(static_cast<long long>(P.B) * P.H, 4ll * num_sms));
  P.combine_smem = 0;
  // the decode's workspace, then the scores
  *score_off = (decode_workspace_bytes(P) + 255) / 256 * 256;
  *ws_bytes = *score_off + static_cast<size_t>(P.B) * P.H * P.max_len * sizeof(float);
  return LRKV_OK;
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_decode_rope_axes_workspace_size(const lrkv_dims* dims, size_t* bytes) {
  if (!bytes) return LRKV_ERR_INVALID_ARG;
  lrkv_status st = lrkv::rope_axes_check(dims);
  if (st != LRKV_OK) return st;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  lrkv::DecodePlan P;
  size_t off = 0;
  return lrkv::rope_axes_plan(*dims, sms, P, &off, bytes);
}

lrkv_status lrkv_decode_rope_axes(const lrkv_dims* dims, const void* q_rot, const void* k_s, const void* v_s,
                                  const void* z_k, const void* z_v, const void* b_k, const void* b_v,
                                  const float* cos_sin, int max_pos, const int32_t* positions, int axes,
                                  const int* sections, const int32_t* seq_lens, float decay, const float* weights,
                                  float* weights_out, float* out, float* lse, void* ws, size_t ws_bytes,
                                  lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_decode_rope_axes");
  lrkv_status st = lrkv::rope_axes_check(dims);
  if (st != LRKV_OK) return st;
  if (!q_rot || !k_s || !v_s || !z_k || !z_v || !b_k || !b_v || !cos_sin || !positions || !seq_lens || !out)
    return LRKV_ERR_INVALID_ARG;
  if (!lrkv::a16(q_rot) || !lrkv::a16(k_s) || !lrkv::a16(v_s) || !lrkv::a16(z_k) || !lrkv::a16(z_v) ||
      !lrkv::a16(b_k) || !lrkv::a16(cos_sin) || !lrkv::a16(out))
    return LRKV_ERR_INVALID_ARG;
  if (max_pos < 1) return LRKV_ERR_INVALID_ARG;
  if (weights_out) {
    if (!lse) return LRKV_ERR_INVALID_ARG;  // the weights need the log-sum-exp
    if ((st = lrkv::weights_check(decay, weights, weights_out)) != LRKV_OK) return st;
  }
  lrkv::AxesArgs A;
  if (!lrkv::rope_axes_make(axes, sections, dims->head_dim, A.ax)) return LRKV_ERR_INVALID_ARG;
  A.positions = positions;
  if (!ws) return LRKV_ERR_WORKSPACE;
  if (!lrkv::a16(ws)) return LRKV_ERR_INVALID_ARG;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  lrkv::DecodePlan P;
  size_t score_off = 0, need = 0;
  if ((st = lrkv::rope_axes_plan(*dims, sms, P, &score_off, &need)) != LRKV_OK) return st;
  if (ws_bytes < need) return LRKV_ERR_WORKSPACE;
  lrkv::decode_bind_workspace(P, ws);
  if (weights_out) P.scores = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + score_off);
  P.q = q_rot; P.k_s = k_s; P.v_s = v_s; P.z_k = z_k; P.z_v = z_v; P.b_k = b_k; P.b_v = b_v;
  P.seq_lens = seq_lens; P.out = out; P.lse = lse;
  P.rope_cs = cos_sin; P.rope_max_pos = max_pos;

  CUtensorMap tm_k, tm_v, tm_zk, tm_zv;
  std::memset(&tm_k, 0, sizeof(tm_k)); std::memset(&tm_v, 0, sizeof(tm_v));
  std::memset(&tm_zk, 0, sizeof(tm_zk)); std::memset(&tm_zv, 0, sizeof(tm_zv));
  const uint64_t row = static_cast<uint64_t>(P.H) * P.r * 2;
  const uint64_t zdims[4] = {static_cast<uint64_t>(P.segw), static_cast<uint64_t>(P.max_len),
                             static_cast<uint64_t>(P.H / P.hs), static_cast<uint64_t>(P.B)};
  const uint64_t zstr[3] = {row, static_cast<uint64_t>(P.segw) * 2, row * P.max_len};
  const uint32_t zbox[4] = {static_cast<uint32_t>(P.segp), static_cast<uint32_t>(lrkv::kRT),
                            static_cast<uint32_t>(P.nsb), 1u};
  if (!lrkv::make_tmap_3d_bf16(&tm_k, k_s, P.dh, P.max_len, P.B, 64, lrkv::kRT, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !lrkv::make_tmap_3d_bf16(&tm_v, v_s, P.dh, P.max_len, P.B, 64, lrkv::kRT, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !lrkv::make_tmap_4d_bf16_strided(&tm_zk, z_k, zdims, zstr, zbox) ||
      !lrkv::make_tmap_4d_bf16_strided(&tm_zv, z_v, zdims, zstr, zbox))
    return LRKV_ERR_CUDA;
  const lrkv::RopeFn kern = lrkv::rope_fn(P.dh, P.r);
  if (lrkv::ensure_kernel_smem(reinterpret_cast<const void*>(kern), P.smem_bytes, true) != cudaSuccess)
    return LRKV_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.grid, P.mt);
  cfg.blockDim = dim3(lrkv::kRThreads);
  cfg.dynamicSmemBytes = P.smem_bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, P, tm_k, tm_v, tm_zk, tm_zv, A) != cudaSuccess) return LRKV_ERR_CUDA;
  if ((st = lrkv::decode_merge_launch(P, stream, true)) != LRKV_OK || !weights_out) return st;
  return lrkv::weights_sum_launch(P.B, P.H, P.max_len, seq_lens, P.scores, lse, decay, weights, weights_out,
                                  stream);
}

}  // extern "C"
