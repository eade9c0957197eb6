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
// from up to `axes` table rows.  Per pair
//   q~ . (k D) = qa (x0 cos - x1 sin) + qb (x0 sin + x1 cos).
//
// The cache's bytes bound it; the rebuild's d_h r multiply-adds per (row, head)
// do so as well when the warps do them (the mma.sync form of this kernel took
// 800 instructions per 16 rows and head, 495 us on 4 x 32K rows of 32 heads).
// So K = Z_h B_h^T runs on tcgen05, 128 rows by d_h columns into one of four
// TMEM accumulators, with a thread per row and half of the pairs behind it: the
// thread keeps its row's cos, sin and shared part in registers for all heads
// of the CTA and spends nine two-wide fp32 instructions on two pairs.  B_h's rows
// are stored in the order x0, x0', x1, x1' of neighbouring pairs, so that two
// pairs' halves lie side by side in TMEM.
//
// Grid (range CTAs, groups of 4 heads), 16 warps: warp 0 copies (TMA: k_s and
// each head's z_k per 128 rows, v_s and z_v per 32 rows), warp 1 issues the
// MMAs, warps 4-11 form the scores (TMEM lane quadrant x half of the pairs; they
// take the registers that the other warps give up), warps 12-15 the softmax and
// the values: each takes a quarter of the shared value
// columns for the four heads and the latents of one head (mma.sync; the
// probabilities as three bf16 parts in free columns of the B operand).
//
// Measured on 4 x 32K rows (32 heads, rank 48): 364 us, the cache at 2.4 TB/s,
// ~12K cycles a tile and CTA where its bytes need 4.6K.  The score warps are at work
// for 93 to 95% of that time, the value warps for 81% (they wait 7% for scores and
// 12% for their copies), each on chains of its own: the scores' gather (positions,
// table entries, the exchange through
// shared memory) takes 3K cycles of a tile and a head's 32 pairs ~2K, the values
// 900 per 16 rows for ten dependent mma.sync.  What was tried and was slower: the
// shared part added by the tensor core (a unit operand, 411 us for 375), TMEM read
// 16 columns ahead of the sums (401 for 375), masks on every tile's values (375).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

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

constexpr int kRT = 128;                     // rows of a tile (TMEM lanes)
constexpr int kRSub = 32;                    // rows of a value copy
constexpr int kRHeads = 4;                   // heads per CTA
constexpr int kRScore = 8;                   // score warps
constexpr int kRValue = 4;                   // value warps
constexpr int kRThreads = 32 * (4 + kRScore + kRValue);
// registers per thread after the split: 512 at most over the four warpgroups, 128 each at launch
constexpr int kRRegsCopy = 56, kRRegsScore = 168, kRRegsValue = 120;
static_assert(kRRegsCopy + 2 * kRRegsScore + kRRegsValue <= 512, "more registers than the block has");
constexpr int kRAcc = 4;                     // TMEM accumulators
constexpr int kRMaxZ = 4, kRMaxV = 8;        // ring depths (at most)
constexpr int kRBox = 16384;                 // 128 rows x 64 columns
constexpr int kRStage = 80;                  // bytes of a row of the gather's staging (64 and a pad)
constexpr float kRRescaleLog2 = 8.f;         // raise the reference max only past 2^8

struct AxesArgs {
  RopeAxes ax;
  int even;                  // 1: no section boundary splits pairs 2 i, 2 i + 1
  const int32_t* positions;  // [B][max_len][axes]
  int nz, nv;                // ring depths: latent boxes, value copies
  int vt_bytes, zv_off;      // bytes of a value copy's slot; offset of its latents
  int off_b, off_k, off_z, off_v, off_st, off_sc, off_q;  // shared memory
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
// 32 lanes x 16 columns of TMEM.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace

template <int DH, int R>
__global__ void __launch_bounds__(kRThreads, 1)
    lrkv_decode_rope_axes_kernel(const __grid_constant__ DecodePlan P, const __grid_constant__ CUtensorMap tm_k,
                                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_zk,
                                 const __grid_constant__ CUtensorMap tm_zv, const __grid_constant__ AxesArgs A) {
  constexpr int NB = DH / 64;        // 64-column boxes of a shared row
  constexpr int HP = DH / 4;         // pairs of a score thread (half of the head's)
  constexpr int MS = DH / 64;        // 16-row tiles of the shared values per value warp
  constexpr int MZ = R / 16;         // 16-row tiles of a head's private values
  constexpr uint32_t kTmemCols = kRAcc * DH;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ uint64_t kfull, kempty, zfull[kRMaxZ], zempty[kRMaxZ], vfull[kRMaxV], vempty[kRMaxV], accf[kRAcc],
      acce[kRAcc], scf[2], sce[2], mdone;
  __shared__ uint32_t tmem_base;
  __shared__ int s_timeout, s_badpos, s_k, s_z, s_v;  // copies issued
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  volatile int* fail = &s_timeout;

  pdl_trigger();  // the merge may launch: it waits for this grid before it reads
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const int B = P.B, H = P.H, h0 = blockIdx.y * kRHeads;
  int* pre = reinterpret_cast<int*>(smem);

  // ---- 1. barriers, TMEM, sequence starts (clamped lengths), B_h -------------------
  if (tid == 0) {
    mbar_init(&kfull, 1);
    mbar_init(&kempty, kRScore);
    for (int i = 0; i < kRMaxZ; ++i) { mbar_init(&zfull[i], 1); mbar_init(&zempty[i], 1); }
    for (int i = 0; i < kRMaxV; ++i) { mbar_init(&vfull[i], 1); mbar_init(&vempty[i], kRValue); }
    for (int i = 0; i < kRAcc; ++i) { mbar_init(&accf[i], 1); mbar_init(&acce[i], kRScore); }
    for (int i = 0; i < 2; ++i) { mbar_init(&scf[i], kRScore); mbar_init(&sce[i], kRValue); }
    mbar_init(&mdone, 1);
    s_timeout = s_badpos = s_k = s_z = s_v = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, kTmemCols);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int N = pre[B];
  const int G = max(1, min(static_cast<int>(gridDim.x), (N + P.min_tokens - 1) / max(P.min_tokens, 1)));
  const int c = blockIdx.x;
  uint32_t* cta_status = P.cta_status + blockIdx.y * gridDim.x + blockIdx.x;
  const bool work = N > 0 && c < G;
  const int g0 = work ? static_cast<int>(static_cast<long long>(c) * N / G) : 0;
  const int g1 = work ? static_cast<int>(static_cast<long long>(c + 1) * N / G) : 0;
  if (work) {
    // row n of head i's operand is B_h's row 4 (n / 4) + {0, 2, 1, 3}[n % 4] (the
    // copy's 128-byte swizzle by hand)
    const __nv_bfloat16* bk = static_cast<const __nv_bfloat16*>(P.b_k) + static_cast<size_t>(h0) * DH * R;
    for (int e = tid; e < kRHeads * DH * (R / 8); e += kRThreads) {
      const int ch = e % (R / 8), n = e / (R / 8) % DH, i = e / (R / 8) / DH;
      const int d = (n & ~3) | ((n & 1) << 1) | ((n >> 1) & 1);
      *reinterpret_cast<uint4*>(smem + A.off_b + (i * DH + n) * 128 + ((ch ^ (n & 7)) << 4)) =
          *reinterpret_cast<const uint4*>(bk + (static_cast<size_t>(i) * DH + d) * R + 8 * ch);
    }
    fence_proxy_async_smem();  // read by the tensor core's own path
  }
  __syncthreads();

  TileWalk w;
  if (!work) {
    // nothing to do
  } else if (warp < 4) {
    regs_down<kRRegsCopy>();
    if (warp == 0 && lane == 0) {
      // ---- copies: the keys' and the values' queues, whichever has a free slot: let go
      // by its readers and, since readers that gave up let go too, landed (a second copy
      // must never join a phase that is still pending; latent slots are let go by the
      // MMAs that read them) -----------------------------------------------------------
      auto again = [&](uint64_t* empty, uint64_t* full, int use) {  // whether use `use` of a slot may begin
        const uint32_t last = static_cast<uint32_t>(use - 1) & 1u;
        return use < 1 || (mbar_test(empty, last) && mbar_test(full, last));
      };
      TileWalk kw, vw;
      bool km = walk_first(kw, pre, B, g0, g1), vm = walk_first(vw, pre, B, g0, g1);
      int kt = 0, ki = 0, zi = 0, vi = 0, vs = 0;  // tile, box within it (0: k_s), boxes, value copies, copy within a tile
      long long idle = clock64();
      while ((km || vm) && !*fail) {
        bool did = false;
        if (km) {
          const int s = zi % A.nz;
          if (ki == 0) {
            if (again(&kempty, &kfull, kt)) {
              mbar_arrive_expect_tx(&kfull, NB * kRBox);
              for (int cb = 0; cb < NB; ++cb)
                tma_load_3d(smem + A.off_k + cb * kRBox, &tm_k, 64 * cb, kw.t0, kw.b, &kfull);
              s_k = ++kt;
              ki = 1;
              did = true;
            }
          } else if (zi < A.nz || mbar_test(&zempty[s], static_cast<uint32_t>(zi / A.nz - 1) & 1u)) {
            mbar_arrive_expect_tx(&zfull[s], kRBox);
            tma_load_4d(smem + A.off_z + s * kRBox, &tm_zk, 0, h0 + ki - 1, kw.t0, kw.b, &zfull[s]);
            s_z = ++zi;
            if (++ki > kRHeads) {
              ki = 0;
              km = walk_next(kw, pre, B, g1, kRT);
            }
            did = true;
          }
        }
        if (vm) {
          const int s = vi % A.nv;
          if (again(&vempty[s], &vfull[s], vi / A.nv)) {
            unsigned char* dst = smem + A.off_v + s * A.vt_bytes;
            mbar_arrive_expect_tx(&vfull[s], NB * kRSub * 128 + P.zt_bytes);
            for (int cb = 0; cb < NB; ++cb)
              tma_load_3d(dst + cb * kRSub * 128, &tm_v, 64 * cb, vw.t0 + vs * kRSub, vw.b, &vfull[s]);
            tma_load_4d(dst + A.zv_off, &tm_zv, 0, vw.t0 + vs * kRSub, blockIdx.y * P.nsb, vw.b, &vfull[s]);
            s_v = ++vi;
            if (++vs * kRSub >= min(kRT, vw.t_end - vw.t0)) {  // copies with rows of the piece only
              vs = 0;
              vm = walk_next(vw, pre, B, g1, kRT);
            }
            did = true;
          }
        }
        if (did) idle = clock64();
        else if (clock64() - idle > P.wait_limit) *fail = 1;
      }
    } else if (warp == 1 && lane == 0) {
      // ---- MMAs: K = Z_h B_h^T of (tile, head) u into accumulator u % 4 ---------------
      constexpr uint32_t idesc = idesc_bf16(128, DH, 0, 0);
      const uint64_t bd = smem_desc(smem_u32(smem + A.off_b), 16, 1024, 2);
      const uint64_t zd = smem_desc(smem_u32(smem + A.off_z), 16, 1024, 2);
      int u = 0;
      bool ok = true;
      for (bool more = walk_first(w, pre, B, g0, g1); more && ok && !*fail; more = walk_next(w, pre, B, g1, kRT))
        for (int i = 0; i < kRHeads; ++i, ++u) {
          const int s = u % A.nz, a = u % kRAcc;
          ok = mbar_wait_bounded(&zfull[s], static_cast<uint32_t>(u / A.nz) & 1u, P.wait_limit) &&
               (u < kRAcc || mbar_wait_bounded(&acce[a], static_cast<uint32_t>(u / kRAcc - 1) & 1u, P.wait_limit));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < R / 16; ++kk)
            tc_mma_ss(tmem + a * DH, zd + static_cast<uint32_t>(s * (kRBox / 16)) + kk * 2,
                      bd + static_cast<uint32_t>(i * DH * 8) + kk * 2, idesc, kk > 0 ? 1u : 0u);
          tc_commit(&zempty[s]);
          tc_commit(&accf[a]);
        }
      tc_commit(&mdone);  // every MMA issued, also by a pass that gave up
      if (!ok) *fail = 1;
    }
  } else if (warp < 4 + kRScore) {
    regs_up<kRRegsScore>();
    // ---- scores: row 32 quad + lane of the tile, pairs half HP .. + HP - 1 -------------
    const int quad = warp & 3, half = (warp - 4) >> 2, row = 32 * quad + lane;
    unsigned char* stage = smem + A.off_st + (warp - 4) * 32 * kRStage;
    float* sq = reinterpret_cast<float*>(smem + A.off_q);              // [4][DH / 4][4]: qa qa' qb qb'
    bool ok = true;
    int cur_b = -1, j = 0, u = 0;
    uint64_t cc[HP / 2], ss[HP / 2];  // cos and sin of pairs 2 i, 2 i + 1 of this thread's half
    int pos[kMaxAxes];
    auto positions_of = [&](const TileWalk& t) {
      const int32_t* at = A.positions + (static_cast<size_t>(t.b) * P.max_len + t.t0 + row) * A.ax.n;
      const bool there = t.t0 + row < t.t_end;
#pragma unroll
      for (int x = 0; x < kMaxAxes; ++x) pos[x] = there && x < A.ax.n ? __ldg(at + x) : 0;
    };
    // byte offsets, 4 bits each, of the axes of this lane's two pairs of every chunk
    uint32_t axis_at = 0u;
#pragma unroll
    for (int ch = 0; ch < HP / 8; ++ch) {
      const int k = half * HP + 8 * ch + 2 * q4;
      axis_at |= static_cast<uint32_t>(4 * A.ax.axis(k) | 4 * A.ax.axis(k + 1) << 4) << (8 * ch);
    }
    bool more = walk_first(w, pre, B, g0, g1);
    if (more) positions_of(w);
    for (; more; ++j) {
      if (w.b != cur_b) {
        cur_b = w.b;
        bar_named(1, 32 * kRScore);  // every score warp is done with the last query
        const __nv_bfloat16* qh = static_cast<const __nv_bfloat16*>(P.q) + (static_cast<size_t>(w.b) * H + h0) * DH;
        for (int e = tid - 128; e < kRHeads * DH / 4; e += 32 * kRScore) {
          const uint2 v = *reinterpret_cast<const uint2*>(qh + 4 * e);
          const float qa = bf_lo(v.x), qb = bf_hi(v.x), ra = bf_lo(v.y), rb = bf_hi(v.y);
          *reinterpret_cast<float4*>(sq + 4 * e) = make_float4(qa, ra, qb, rb);
        }
        bar_named(1, 32 * kRScore);
      }
      // the rotations, 8 pairs of the warp's 32 rows at a time: 4 lanes load a row's
      // 64 bytes, the row's own lane takes them from shared memory
#pragma unroll
      for (int x = 0; x < kMaxAxes; ++x) {
        if (pos[x] < 0 || pos[x] >= P.rope_max_pos) {
          s_badpos = 1;
          pos[x] = min(max(pos[x], 0), P.rope_max_pos - 1);
        }
      }
      __syncwarp();
      *reinterpret_cast<int4*>(stage + lane * kRStage) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      __syncwarp();
      float4 e[HP / 8][4];
      const float* table = P.rope_cs + 2 * (half * HP + 2 * q4);  // this lane's two pairs of chunk 0
      if (A.even) {
#pragma unroll
        for (int ch = 0; ch < HP / 8; ++ch) {
          const unsigned char* pa = stage + g * kRStage + (axis_at >> (8 * ch) & 0xfu);
#pragma unroll
          for (int r8 = 0; r8 < 4; ++r8)
            e[ch][r8] = __ldg(reinterpret_cast<const float4*>(
                table + static_cast<size_t>(*reinterpret_cast<const int*>(pa + 8 * r8 * kRStage)) * DH + 16 * ch));
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < HP / 8; ++ch) {
          const unsigned char* pa = stage + g * kRStage + (axis_at >> (8 * ch) & 0xfu);
          const unsigned char* pb = stage + g * kRStage + (axis_at >> (8 * ch + 4) & 0xfu);
#pragma unroll
          for (int r8 = 0; r8 < 4; ++r8) {
            const size_t ra = static_cast<size_t>(*reinterpret_cast<const int*>(pa + 8 * r8 * kRStage)) * DH;
            const size_t rb = static_cast<size_t>(*reinterpret_cast<const int*>(pb + 8 * r8 * kRStage)) * DH;
            const float2 a = __ldg(reinterpret_cast<const float2*>(table + ra + 16 * ch));
            const float2 b = __ldg(reinterpret_cast<const float2*>(table + rb + 16 * ch + 2));
            e[ch][r8] = make_float4(a.x, a.y, b.x, b.y);
          }
        }
      }
      // (the next tile's positions load meanwhile)
      more = walk_next(w, pre, B, g1, kRT);
      if (more) positions_of(w);
#pragma unroll
      for (int ch = 0; ch < HP / 8; ++ch) {
        __syncwarp();
#pragma unroll
        for (int r8 = 0; r8 < 4; ++r8)
          *reinterpret_cast<float4*>(stage + (8 * r8 + g) * kRStage + 16 * q4) =
              make_float4(e[ch][r8].x, e[ch][r8].z, e[ch][r8].y, e[ch][r8].w);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(stage + lane * kRStage + 16 * i);
          cc[4 * ch + i] = v.x;
          ss[4 * ch + i] = v.y;
        }
      }
      // the row's shared part, two columns per word
      ok = ok && !*fail && mbar_wait_bounded(&kfull, static_cast<uint32_t>(j) & 1u, P.wait_limit);
      ok = __all_sync(0xffffffffu, ok);
      uint32_t sk[HP];
      if (ok) {
        const unsigned char* kr = smem + A.off_k + (DH == 128 ? half * kRBox : 0) + row * 128;
#pragma unroll
        for (int i = 0; i < HP / 4; ++i) {
          const int chunk = (DH == 128 ? 0 : half * (HP / 4)) + i;
          const uint4 v = *reinterpret_cast<const uint4*>(kr + ((chunk ^ (row & 7)) << 4));
          sk[4 * i] = v.x; sk[4 * i + 1] = v.y; sk[4 * i + 2] = v.z; sk[4 * i + 3] = v.w;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&kempty);
      // the score buffer of tile j - 2 is free
      ok = ok && (j < 2 || mbar_wait_bounded(&sce[j & 1], static_cast<uint32_t>(j / 2 - 1) & 1u, P.wait_limit));
      float* sc = reinterpret_cast<float*>(smem + A.off_sc) + ((j & 1) * 2 + half) * kRHeads * kRT + row;
#pragma unroll 1
      for (int i = 0; i < kRHeads; ++i, ++u) {
        const int a = u % kRAcc;
        ok = ok && !*fail && mbar_wait_bounded(&accf[a], static_cast<uint32_t>(u / kRAcc) & 1u, P.wait_limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          *fail = 1;
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&acce[a]);
          continue;
        }
        tc_fence_after();
        const uint32_t at = tmem + (static_cast<uint32_t>(32 * quad) << 16) + a * DH + half * (DH / 2);
        const float* qa = sq + i * DH + half * (DH / 2);
        uint64_t acc0 = 0ull, acc1 = 0ull, acc2 = 0ull;  // qa x0 cos, qb (x0 sin + x1 cos), qa x1 sin
        uint32_t v[DH / 32][16];
#pragma unroll
        for (int c16 = 0; c16 < DH / 32; c16 += 2) {
          tmem_ld16(at + 16 * c16, v[c16]);
          tmem_ld16(at + 16 * c16 + 16, v[c16 + 1]);
          tmem_wait_ld();
          if (c16 + 2 == DH / 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cta(&acce[a]);  // the accumulator is free
          }
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const int dp = 4 * c16 + p;  // pairs 2 dp, 2 dp + 1 of the half
            const uint32_t* x = &v[c16 + p / 4][4 * (p & 3)];
            const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(qa + 4 * dp);
            const uint32_t sa = sk[2 * dp], sb = sk[2 * dp + 1];
            const uint64_t x0 = add2(pair(__uint_as_float(x[0]), __uint_as_float(x[1])), pair(bf_lo(sa), bf_lo(sb)));
            const uint64_t x1 = add2(pair(__uint_as_float(x[2]), __uint_as_float(x[3])), pair(bf_hi(sa), bf_hi(sb)));
            acc0 = fma2(qv.x, mul2(cc[dp], x0), acc0);
            acc2 = fma2(qv.x, mul2(ss[dp], x1), acc2);
            acc1 = fma2(qv.y, fma2(ss[dp], x0, mul2(cc[dp], x1)), acc1);
          }
        }
        {
          float u0, u1, v0, v1;
          unpair(acc0, u0, u1);
          unpair(acc2, v0, v1);
          acc0 = pair(u0 - v0, u1 - v1);
        }
        float a0, a1, b0, b1;
        unpair(acc0, a0, a1);
        unpair(acc1, b0, b1);
        sc[i * kRT] = (a0 + a1) + (b0 + b1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&scf[j & 1]);
    }
    if (!ok) *fail = 1;
  } else {
    regs_down<kRRegsValue>();
    // ---- softmax and values: shared columns 16 MS v .. of the four heads, latents of
    // head v -----------------------------------------------------------------------
    const int v = warp - 4 - kRScore, hd = g & 3;  // this lane's softmax: head hd
    const int trow = (lane & 7) + 8 * (lane >> 4), tcol = (lane >> 3) & 1;
    const int zoff = (v / P.hs) * (kRSub * P.segp * 2) + (v % P.hs) * R * 2;
    pdl_wait();  // the launch before may still read the workspace
    bool ok = true;
    int cur_b = -1, j = 0, vi = 0;
    float m = -INFINITY, l = 0.f;
    // columns 0-3 the heads' high and third parts, 4-7 their low parts (of oz
    // only head v's two columns mean anything)
    float os[MS][4], oz[MZ][4];
    // the tensor cores cut each sum short of fp32 rounding (1e-5 off after 800
    // steps): a tile's products get accumulators of their own
    float ts[MS][4], tz[MZ][4];
    auto write_partial = [&](int b) {
      const size_t slot = static_cast<size_t>(b + c);
      float lsum = l;
      lsum += __shfl_xor_sync(0xffffffffu, lsum, 1);
      lsum += __shfl_xor_sync(0xffffffffu, lsum, 2);
      if (lane == 4 * v) {
        float* pml = P.part_ml + (slot * H + h0 + v) * 2;
        pml[0] = m;
        pml[1] = lsum;
      }
#pragma unroll
      for (int e = 0; e < MS; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) os[e][k] += __shfl_xor_sync(0xffffffffu, os[e][k], 2);
#pragma unroll
      for (int e = 0; e < MZ; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) oz[e][k] += __shfl_xor_sync(0xffffffffu, oz[e][k], 2);
      if (q4 < 2) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float* o = P.part_acc + (slot * H + h0 + 2 * q4 + x) * (DH + R) + 16 * MS * v;
#pragma unroll
          for (int e = 0; e < MS; ++e) {
            o[16 * e + g] = os[e][x];
            o[16 * e + g + 8] = os[e][2 + x];
          }
        }
      }
      if (q4 == v >> 1) {
        float* o = P.part_acc + (slot * H + h0 + v) * (DH + R) + DH;
#pragma unroll
        for (int e = 0; e < MZ; ++e) {
          o[16 * e + g] = (v & 1) ? oz[e][1] : oz[e][0];
          o[16 * e + g + 8] = (v & 1) ? oz[e][3] : oz[e][2];
        }
      }
    };
    bool more = walk_first(w, pre, B, g0, g1);
    for (; more; ++j) {
      if (w.b != cur_b) {
        if (cur_b >= 0) write_partial(cur_b);
        cur_b = w.b;
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < MS; ++e) os[e][0] = os[e][1] = os[e][2] = os[e][3] = 0.f;
#pragma unroll
        for (int e = 0; e < MZ; ++e) oz[e][0] = oz[e][1] = oz[e][2] = oz[e][3] = 0.f;
      }
      const int nvalid = min(kRT, w.t_end - w.t0);
      ok = ok && !*fail && mbar_wait_bounded(&scf[j & 1], static_cast<uint32_t>(j / 2) & 1u, P.wait_limit);
      ok = __all_sync(0xffffffffu, ok);
      float s[32];  // scores of head hd: s[4 t + {0, 1, 2, 3}] rows 16 t + 2 q4 + {0, 1, 8, 9}
      if (ok) {
        const float* lo = reinterpret_cast<const float*>(smem + A.off_sc) + (j & 1) * 2 * kRHeads * kRT;
        const float* hi = lo + kRHeads * kRT;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = 16 * t + 8 * k + 2 * q4;
            const float2 a = *reinterpret_cast<const float2*>(lo + hd * kRT + r);
            const float2 b = *reinterpret_cast<const float2*>(hi + hd * kRT + r);
            s[4 * t + 2 * k] = r < nvalid ? (a.x + b.x) * P.scale_log2 : -INFINITY;
            s[4 * t + 2 * k + 1] = r + 1 < nvalid ? (a.y + b.y) * P.scale_log2 : -INFINITY;
          }
        if (P.scores) {
          float* out = P.scores + (static_cast<size_t>(w.b) * H + h0 + v) * P.max_len + w.t0;
#pragma unroll
          for (int k = 0; k < kRT / 32; ++k) {
            const int r = 32 * k + lane;
            if (r < nvalid) out[r] = (lo[v * kRT + r] + hi[v * kRT + r]) * P.scale_log2;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&sce[j & 1]);
      if (ok) {
        // one online softmax per head (log2 domain), the reference raised lazily
        float mx = s[0];
#pragma unroll
        for (int k = 1; k < 32; ++k) mx = fmaxf(mx, s[k]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const bool up = mx > m + kRRescaleLog2;
        if (__any_sync(0xffffffffu, up)) {
          const float alpha = !up ? 1.f : m == -INFINITY ? 0.f : exp2f(m - mx);
          if (up) m = mx;
          l *= alpha;
          const float a0 = __shfl_sync(0xffffffffu, alpha, 4 * ((2 * q4) & 3));  // columns 2 q4, 2 q4 + 1
          const float a1 = __shfl_sync(0xffffffffu, alpha, 4 * ((2 * q4 + 1) & 3));
#pragma unroll
          for (int e = 0; e < MS; ++e) {
            os[e][0] *= a0; os[e][1] *= a1; os[e][2] *= a0; os[e][3] *= a1;
          }
#pragma unroll
          for (int e = 0; e < MZ; ++e) {
            oz[e][0] *= a0; oz[e][1] *= a1; oz[e][2] *= a0; oz[e][3] *= a1;
          }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          s[k] = exp2f(s[k] - m);
          l += s[k];
        }
      }
#pragma unroll
      for (int e = 0; e < MS; ++e) ts[e][0] = ts[e][1] = ts[e][2] = ts[e][3] = 0.f;
#pragma unroll
      for (int e = 0; e < MZ; ++e) tz[e][0] = tz[e][1] = tz[e][2] = tz[e][3] = 0.f;
      auto products = [&](auto masked) {
        constexpr bool M = decltype(masked)::value;
#pragma unroll
        for (int sub = 0; sub < kRT / kRSub; ++sub) {
          if (sub * kRSub >= nvalid) break;
          const int slot = vi % A.nv;
          ok = ok && !*fail && mbar_wait_bounded(&vfull[slot], static_cast<uint32_t>(vi / A.nv) & 1u, P.wait_limit);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            const unsigned char* vsm = smem + A.off_v + slot * A.vt_bytes;
            const unsigned char* zsm = vsm + A.zv_off + zoff;
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {
              const int t = 2 * sub + t2;  // 16 rows
              // three bf16 parts of the probabilities of rows 2 q4, + 1 (first word), + 8, + 9 (second)
              uint32_t p1[2], p2[2], p3[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float x = s[4 * t + 2 * k], y = s[4 * t + 2 * k + 1];
                p1[k] = pack_bf16(x, y);
                const float x2 = x - bf_lo(p1[k]), y2 = y - bf_hi(p1[k]);
                p2[k] = pack_bf16(x2, y2);
                p3[k] = pack_bf16(x2 - bf_lo(p2[k]), y2 - bf_hi(p2[k]));
              }
              // column g: the high part of head g, the low part of head g - 4; then the third parts
              const uint32_t b0 = g < 4 ? p1[0] : p2[0], b1 = g < 4 ? p1[1] : p2[1];
              const uint32_t c0 = g < 4 ? p3[0] : 0u, c1 = g < 4 ? p3[1] : 0u;
              // rows past the piece (which may hold anything) must not meet their
              // zero probabilities as 0 x NaN
              const int left = nvalid - 16 * t;
              const uint32_t k0 = !M ? 0u : (2 * q4 < left ? 0x0000ffffu : 0u) | (2 * q4 + 1 < left ? 0xffff0000u : 0u);
              const uint32_t k1 =
                  !M ? 0u : (2 * q4 + 8 < left ? 0x0000ffffu : 0u) | (2 * q4 + 9 < left ? 0xffff0000u : 0u);
              const int r = 16 * t2 + trow;
#pragma unroll
              for (int e = 0; e < MS; ++e) {
                uint32_t x0, x1, x2, x3;
                const int ch = 2 * (MS * v + e) + tcol;  // 16-byte chunk along the head dim
                ldsm_x4_trans(x0, x1, x2, x3, vsm + (ch >> 3) * (kRSub * 128) + swz_off(r, ch & 7, 128));
                if (M) {
                  x0 &= k0; x1 &= k0; x2 &= k1; x3 &= k1;
                }
                mma_bf16_16816(ts[e], x0, x1, x2, x3, b0, b1);
                mma_bf16_16816(ts[e], x0, x1, x2, x3, c0, c1);
              }
#pragma unroll
              for (int e = 0; e < MZ; ++e) {
                uint32_t x0, x1, x2, x3;
                ldsm_x4_trans(x0, x1, x2, x3, zsm + r * (P.segp * 2) + (16 * e + 8 * tcol) * 2);
                if (M) {
                  x0 &= k0; x1 &= k0; x2 &= k1; x3 &= k1;
                }
                mma_bf16_16816(tz[e], x0, x1, x2, x3, b0, b1);
                mma_bf16_16816(tz[e], x0, x1, x2, x3, c0, c1);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cta(&vempty[slot]);
          ++vi;
        }
      };
      if (nvalid < kRT)
        products(std::true_type{});
      else
        products(std::false_type{});
#pragma unroll
      for (int e = 0; e < MS; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) os[e][k] += ts[e][k];
#pragma unroll
      for (int e = 0; e < MZ; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) oz[e][k] += tz[e][k];
      more = walk_next(w, pre, B, g1, kRT);
    }
    if (cur_b >= 0) write_partial(cur_b);
    if (!ok) *fail = 1;
  }

  // ---- every copy and MMA this CTA issued is complete before it exits ----
  __syncthreads();
  if (tid == 0) {
    bool done = true;
    if (s_k > 0) done = mbar_wait_bounded(&kfull, static_cast<uint32_t>(s_k - 1) & 1u);
    for (int i = max(0, s_z - A.nz); i < s_z; ++i)
      done = mbar_wait_bounded(&zfull[i % A.nz], static_cast<uint32_t>(i / A.nz) & 1u) && done;
    for (int i = max(0, s_v - A.nv); i < s_v; ++i)
      done = mbar_wait_bounded(&vfull[i % A.nv], static_cast<uint32_t>(i / A.nv) & 1u) && done;
    if (work) done = mbar_wait_bounded(&mdone, 0u) && done;
    if (!done) *fail = 1;
    pdl_wait();  // the launch before may still read the workspace
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      P.meta[0] = N;
      P.meta[1] = G;
    }
    *cta_status = (bad || s_badpos ? kDevBounds : 0u) | (*fail ? kDevTimeout : 0u);
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    pdl_wait();
    for (int b = tid; b <= B; b += blockDim.x) P.prefix[b] = pre[b];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
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
  if (d->dtype != LRKV_BF16 || !rope_fn(d->head_dim, d->rank) || d->heads % 8 != 0) return LRKV_ERR_UNSUPPORTED;
  if (d->batch > kMaxBatch || static_cast<long long>(d->batch) * d->max_len > (1LL << 31) - 1)
    return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

lrkv_status rope_axes_plan(const lrkv_dims& d, int num_sms, DecodePlan& P, AxesArgs& A, size_t* score_off,
                           size_t* ws_bytes) {
  std::memset(&P, 0, sizeof(P));
  std::memset(&A, 0, sizeof(A));
  P.B = d.batch; P.H = d.heads; P.dh = d.head_dim; P.r = d.rank; P.max_len = d.max_len;
  P.map_len = d.max_len; P.map_seqs = d.batch;
  const float scale = d.scale > 0.f ? d.scale : 1.f / std::sqrt(static_cast<float>(d.head_dim));
  P.scale_log2 = scale * kLog2e;
  P.bf16 = 1; P.esz = 2; P.T = kRT; P.stream = 1;
  P.wait_limit = wait_limit_cycles();
  P.mt = P.H / kRHeads;
  P.grid = std::max(1, num_sms / P.mt);
  P.ngw = 1;
  // value latents: segments of hs heads, rows padded to an odd number of 16-byte chunks
  P.hs = 4 * P.r + 8 <= 256 ? 4 : 2;
  P.segw = P.hs * P.r;
  P.segp = P.segw + 8;
  P.nsb = kRHeads / P.hs;
  P.zt_bytes = P.nsb * kRSub * P.segp * 2;
  // shared memory: sequence starts | B_h | k_s | latent ring | value ring | staging | scores | queries;
  // the value ring takes what is left
  const int nb = P.dh / 64;
  A.zv_off = nb * kRSub * 128;
  A.vt_bytes = round_up(A.zv_off + P.zt_bytes, 1024);
  const int budget = 224 * 1024;  // (3 KB of the 227 for the static part and the alignment)
  const int fixed = round_up((P.B + 1) * 4, 1024) + kRHeads * P.dh * 128 + nb * kRBox + kRScore * 32 * kRStage +
                    2 * 2 * kRHeads * kRT * 4 + kRHeads * P.dh * 4;
  for (A.nz = 3; A.nz >= 1; --A.nz) {
    A.nv = std::min(kRMaxV, (budget - fixed - A.nz * kRBox) / A.vt_bytes);
    if (A.nv >= 2) break;
  }
  if (A.nz < 1) return LRKV_ERR_UNSUPPORTED;
  int off = round_up((P.B + 1) * 4, 1024);
  A.off_b = off; off += kRHeads * P.dh * 128;
  A.off_k = off; off += nb * kRBox;
  A.off_z = off; off += A.nz * kRBox;
  A.off_v = off; off += A.nv * A.vt_bytes;
  A.off_st = off; off += kRScore * 32 * kRStage;
  A.off_sc = off; off += 2 * 2 * kRHeads * kRT * 4;
  A.off_q = off; off += kRHeads * P.dh * 4;
  P.smem_bytes = off + 1024;
  P.min_tokens = kRT;
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
  lrkv::AxesArgs A;
  size_t off = 0;
  return lrkv::rope_axes_plan(*dims, sms, P, A, &off, bytes);
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
  lrkv::RopeAxes ax;
  if (!lrkv::rope_axes_make(axes, sections, dims->head_dim, ax)) return LRKV_ERR_INVALID_ARG;
  if (!ws) return LRKV_ERR_WORKSPACE;
  if (!lrkv::a16(ws)) return LRKV_ERR_INVALID_ARG;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  lrkv::DecodePlan P;
  lrkv::AxesArgs A;
  size_t score_off = 0, need = 0;
  if ((st = lrkv::rope_axes_plan(*dims, sms, P, A, &score_off, &need)) != LRKV_OK) return st;
  if (ws_bytes < need) return LRKV_ERR_WORKSPACE;
  lrkv::decode_bind_workspace(P, ws);
  if (weights_out) P.scores = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + score_off);
  P.q = q_rot; P.k_s = k_s; P.v_s = v_s; P.z_k = z_k; P.z_v = z_v; P.b_k = b_k; P.b_v = b_v;
  P.seq_lens = seq_lens; P.out = out; P.lse = lse;
  P.rope_cs = cos_sin; P.rope_max_pos = max_pos;
  A.ax = ax;
  A.positions = positions;
  A.even = 1;
  for (int a = 0; a < axes; ++a) A.even = A.even && ax.end[a] % 2 == 0;

  CUtensorMap tm_k, tm_v, tm_zk, tm_zv;
  std::memset(&tm_k, 0, sizeof(tm_k)); std::memset(&tm_v, 0, sizeof(tm_v));
  std::memset(&tm_zk, 0, sizeof(tm_zk)); std::memset(&tm_zv, 0, sizeof(tm_zv));
  const uint64_t r = P.r, H = P.H, L = P.max_len, B = P.B;
  const uint64_t kdims[4] = {r, H, L, B}, kstr[3] = {r * 2, H * r * 2, L * H * r * 2};
  const uint32_t kbox[4] = {64u, 1u, static_cast<uint32_t>(lrkv::kRT), 1u};
  const uint64_t vdims[4] = {static_cast<uint64_t>(P.segw), L, H / P.hs, B};
  const uint64_t vstr[3] = {H * r * 2, static_cast<uint64_t>(P.segw) * 2, L * H * r * 2};
  const uint32_t vbox[4] = {static_cast<uint32_t>(P.segp), static_cast<uint32_t>(lrkv::kRSub),
                            static_cast<uint32_t>(P.nsb), 1u};
  if (!lrkv::make_tmap_3d_bf16(&tm_k, k_s, P.dh, L, B, 64, lrkv::kRT, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !lrkv::make_tmap_3d_bf16(&tm_v, v_s, P.dh, L, B, 64, lrkv::kRSub, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !lrkv::make_tmap_4d_bf16_swizzled(&tm_zk, z_k, kdims, kstr, kbox) ||
      !lrkv::make_tmap_4d_bf16_strided(&tm_zv, z_v, vdims, vstr, vbox))
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
