// decode8.cu — one decode step over the factored cache in 8 bits
// (lrkv_decode8): every element is an e4m3 number times the scale of its block
// of 16 rows and head.
//
//   score_{h,j} = (ks_j (q_h . k8_j) + kz_{j,h} (p_h . z8_{j,h})) scale,  p_h = q_h B_h^K
//   o_h = sum_j a_{h,j} vs_j v8_j + (sum_j a_{h,j} vz_{j,h} z8_{j,h}) (B_h^V)^T
//
// The cache's bytes bound it, so they go from memory to the tensor cores as
// they are: TMA lays 128 rows x 128 columns boxes down, tcgen05.mma (kind
// f8f6f4) takes them as its A operand, K-major (rows as M) for the scores,
// MN-major (columns as M, rows as K) for the values.  What multiplies them is
// fp32 (p, the probabilities) or bf16 (q), and is split into e4m3 parts, each
// the rounding of what the ones before left, times 16: four significant bits a
// part, six parts for fp32, four for q.  The parts are columns of the B
// operand; a product of 128 x N x 32 costs the same 46 cycles for every N up
// to 48, so the parts of eight heads cost what one column would.  The part
// sums come back from TMEM and are added in fp32.  A tile's products start
// from zero, so that the tensor core's truncation (2^-21 of the sum of the
// magnitudes at worst) does not grow with the length; the sums over the tiles
// are in registers.
//
// Heads go in groups of eight, a CTA each; the latents of a group are a block
// diagonal operand (zero columns for the other heads).  The shared rows are read
// by every group; all but the first find them in L2.
//
// Grid (range CTAs, groups).  16 warps: 0-7 the softmax (a thread per row, four
// heads each), 8-11 the value sums (a thread per column), 12 and 15 the copies
// (keys, with the operands of each sequence, which lrkv_decode8_operands_kernel
// has laid out before; values), 13 the score MMAs, 14 the value MMAs.  Keys and
// values have a ring each, so that each has one warp that fills and one that
// frees it: with two of either a barrier's parity could be two phases old.  The
// scores of the next tile are formed while the softmax works on this one.
//
// Each CTA has an equal part of all tiles.  A sequence that several CTAs share is
// joined by the last of them to be done with it, in the order of its pieces;
// results do not depend on which one that is.  (With a merge kernel behind the
// scan a call took 21 us of the host's time instead of 13.)
//
// Measured on GB300, back-to-back calls of a graph, scales read along with the
// cache: 4 x 65,536 rows of 32 heads, rank 48, d_h 128: 135-139 us, 6.3-6.5 TB/s
// (0.95-0.97 of a measured copy's 6.7); 32 x 1-8K rows in pages of 256, rank 56:
// 101-103 us, 5.5 TB/s; 8 x 4096 rows, 16 heads, rank 28, d_h 64: 17.2 us, 2 TB/s;
// one sequence of 517 rows: 10.4 us.  The long scans are bound by memory; what the
// others take beside it is latency: 3-4 us until the first operands are there, 2 us
// from the last product to knowing who joins, 2-3 us for a join.
//
// Slower, and not taken: latents marked evict-first in L2 (4 x 65,536 rows: 154 us for 145 then), operands formed by
// each CTA of the scan, which then need not wait for the launch before (28 us for 19 on 8 x 4096 rows: the CTAs drift
// apart and no longer find the shared rows in L2), B_h^V fetched in part or whole only once it is known who joins
// (10.5 us for 10.2, 137.7 for 137.5).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache8.h"
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

constexpr int k8Rows = 128;        // rows of a tile, the step of the split
constexpr int k8Step = 32;         // rows of a K step of the value products
constexpr int k8Heads = 8;         // heads of a CTA
constexpr int k8QParts = 4, k8Parts = 6;
constexpr int k8NQ = k8Heads * k8QParts, k8N = k8Heads * k8Parts;  // columns of the operands
constexpr int k8Box = 16384;       // 128 rows x 128 columns
constexpr int k8MaxSlots = 14;
constexpr int k8Softmax = 8, k8Values = 4;
constexpr int k8Threads = 32 * (k8Softmax + k8Values + 4);
constexpr int k8MaxD = 2, k8MaxZ = 4;  // 128-column chunks of a shared row, of a group's latents
// TMEM columns: two score buffers, then the value products
constexpr uint32_t k8S = 0, k8SWidth = k8NQ + k8N, k8Os = 2 * k8SWidth, k8Oz = k8Os + k8MaxD * k8N, k8Cols = 512;
static_assert(k8Oz + k8MaxZ * k8N <= k8Cols, "more TMEM than there is");

// Maps of the cache's tensors: k_s, v_s, z_k, z_v with boxes of Args8::box rows, then of tail_box rows.
struct Maps8 {
  CUtensorMap map[8];
};

struct Args8 {
  int B, H, dh, r, max_len;
  float scale_log2;     // scale * log2(e): scores live in the base-2 domain
  long long wait_limit; // SM cycles a wait may take before it gives up
  int groups, nd, nz;   // head groups; chunks of a shared row and of a group's latents
  int img_bytes;        // operands of a (sequence, group): q parts | p parts | 16 factors
  int img_pad;          // the same in shared memory, on a 1 KB boundary
  int slots[2];         // ring depths: keys, values
  int box, tail_box;    // rows of a copy: of a full tile (128, or a page's), of a sequence's last one (32, or a page's)
  int off_img, off_p, off_ring, smem_bytes;
  int blocks;           // scale blocks of a sequence (contiguous) or page
  int grid;             // range CTAs of a group
  // the join: columns of b_v a copy takes (its alignment), heads lifted at once (shared memory), bytes of a row there
  int vec, lift, pitch;
  const int32_t* block_table;  // [B][max_blocks] or NULL (contiguous)
  int max_blocks, page_shift, num_pages;
  const void *q, *b_k, *b_v;
  const int32_t* seq_lens;
  float *out, *lse;
  lrkv_cache8 cache;
  // workspace
  uint32_t* status;
  int* arrived;           // [B][groups] range CTAs done with a sequence
  float* part_ml;         // [B + grid][H][2] maxima (log2 domain) and denominators of the pieces
  float* part_acc;        // [B + grid][H][dh + r] their sums of shared values and latents
  unsigned char* images;  // [B][groups][img_bytes]
};

__device__ __forceinline__ void mma8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// e4m3 A and B, fp32 D, M = 128; mn: A and B are MN-major.
__host__ __device__ constexpr uint32_t idesc8(int N, int mn) {
  return (1u << 4) | (static_cast<uint32_t>(mn) << 15) | (static_cast<uint32_t>(mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t* v) {
  static_assert(N == 16 || N == 8 || N == 4 || N == 2, "");
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(t));
  else if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(t));
  else if constexpr (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(t));
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(t));
}
// Sum of N part sums, each worth a 16th of the one before.
template <int N>
__device__ __forceinline__ float join(const uint32_t* v) {
  float s = __uint_as_float(v[N - 1]);
#pragma unroll
  for (int i = N - 2; i >= 0; --i) s = fmaf(s, 0.0625f, __uint_as_float(v[i]));
  return s;
}
// The probabilities' operand, MN-major without swizzle: 16 columns of a row are 16 bytes, 8 rows a core matrix,
// the three groups of 16 columns follow each other, then the next 8 rows.  A thread writes four heads of a row:
// parts 0-3 of the first (second) four heads are group 0 (1), parts 4-5 of all the last group.
constexpr int k8PGroup = 128, k8PRows = 3 * k8PGroup, k8PBytes = k8Rows / 8 * k8PRows;
// The six part sums of head k of four, of which `v` holds the first 16 columns and `w` the last 8.
__device__ __forceinline__ float join_values(const uint32_t* v, const uint32_t* w, int k) {
  float s = fmaf(__uint_as_float(w[4 + k]), 0.0625f, __uint_as_float(w[k]));
#pragma unroll
  for (int i = 3; i >= 0; --i) s = fmaf(s, 0.0625f, __uint_as_float(v[4 * i + k]));
  return s;
}
// 2^-e of x in [2^e, 2^(e + 1)) (0: 2^127), and 2^e (0: 0), of numbers far from the ends of fp32's range.
__device__ __forceinline__ float down_to_one(float x) {
  return __uint_as_float(0x7f000000u - (__float_as_uint(x) & 0x7f800000u));
}
__device__ __forceinline__ float power_in(float x) { return __uint_as_float(__float_as_uint(x) & 0x7f800000u); }
// m in [1, 2) and a whole number e with x = m 2^e, of any positive finite x (subnormal ones too); 0: m = 0, e = -191.
// Through a power of two that makes x normal and 2^-e representable.
__device__ __forceinline__ float split_scale(float x, float& e) {
  const bool small = x < 1.f;
  const float y = x * (small ? 0x1p64f : 0x1p-64f);
  const uint32_t u = __float_as_uint(y);
  e = __uint_as_float(0x4b000000u | u >> 23) - (small ? 0x1p23f + 191.f : 0x1p23f + 63.f);  // (2^23 + the field, exact)
  return y * __uint_as_float(0x7f000000u - (u & 0x7f800000u));
}
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_min(float v) {
  float r;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Waits for a phase unless the CTA has given up, and gives up itself at the bound.  (A try may last as long as the
// hardware likes, a few microseconds: bounds below that are polled.)
__device__ __forceinline__ bool wait8(uint64_t* bar, uint32_t parity, volatile int* fail, long long limit) {
  auto done = [&] { return limit > 100000 ? mbar_try_wait(bar, parity) : mbar_test(bar, parity); };
  if (done()) return true;
  const long long t0 = clock64();
  while (!done()) {
    if (*fail) return false;
    if (clock64() - t0 > limit) {
      *fail = 1;
      return false;
    }
  }
  return true;
}
// The same by a whole warp.
__device__ __forceinline__ bool wait8_warp(uint64_t* bar, uint32_t parity, volatile int* fail, long long limit) {
  const bool ok = wait8(bar, parity, fail, limit);
  return __all_sync(0xffffffffu, ok);
}
// A place in the ring: a slot, and the phase of its barriers.
struct Place8 {
  int slot = 0;
  uint32_t phase = 0u;
  __device__ __forceinline__ void move(int n, int slots) {  // n <= slots
    slot += n;
    if (slot >= slots) {
      slot -= slots;
      phase ^= 1u;
    }
  }
};
// `steps` (1 .. 4) MMAs of K = 32 along a box and an operand.
__device__ __forceinline__ void mma8_box(uint32_t d, uint64_t a, int a_step, uint64_t b, int b_step, uint32_t idesc,
                                         int steps, bool fresh) {
  mma8(d, a, b, idesc, fresh ? 0u : 1u);
  if (steps == 4) {
    mma8(d, a + a_step, b + b_step, idesc, 1u);
    mma8(d, a + 2 * a_step, b + 2 * b_step, idesc, 1u);
    mma8(d, a + 3 * a_step, b + 3 * b_step, idesc, 1u);
  } else {
    for (int k = 1; k < steps; ++k) mma8(d, a + k * a_step, b + k * b_step, idesc, 1u);
  }
}
// The copying and issuing warps run as whole warps on values that every lane has, so that the operands of their
// instructions are in uniform registers: with one lane's own values each MMA took three times as long to issue.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}
// The pieces of a CTA's range of tiles [g0, g1): tiles [t0, t0 + n) of sequence b.
struct Pieces8 {
  int b, g, t0, n;
  __device__ __forceinline__ bool first(const int* pre, int B, int g0, int g1) {
    TileWalk w;
    if (!walk_first(w, pre, B, g0, g1)) return false;
    b = uniform(w.b);
    g = uniform(g0);
    t0 = uniform(w.t0);
    n = uniform(w.t_end) - t0;
    return true;
  }
  __device__ __forceinline__ bool next(const int* pre, int B, int g1) {
    g += n;
    if (g >= uniform(g1)) return false;
    do ++b; while (uniform(pre[b + 1]) <= g);  // (empty sequences)
    t0 = 0;
    n = uniform(min(pre[b + 1], g1)) - g;
    return true;
  }
};
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace

// ============================================================== the operands
// One CTA per (head, sequence): p = q B^K in fp32, then q and p as e4m3 parts
// in the layout of the MMA's B operand (K-major, 128-byte swizzle): row
// (head, part), a byte per column, zeros in the columns of the other heads.
// Both are brought to a largest magnitude in [128, 256) first; the factors
// undo that and hold the scale (log2 domain).
// Latency is all it costs (B_h^K once per sequence, from L2): the words of B_h^K
// are under way before q is.
constexpr int k8OpWarps = 8, k8OpThreads = 32 * k8OpWarps;
static_assert(k8MaxD * 128 <= k8OpThreads && k8MaxZ * 128 <= 2 * k8OpThreads, "a thread's columns");
constexpr int k8OpRows = 16;  // rows of B_h^K a warp has in flight

__global__ void __launch_bounds__(k8OpThreads) lrkv_decode8_operands_kernel(const __grid_constant__ Args8 A) {
  __shared__ float s_q[256], s_part[k8OpWarps][64];
  __shared__ uint32_t s_max[2][k8OpWarps];
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, hl = h & 7, d = A.dh, r = A.r;
  const bool there = h < A.H;
  // lanes hold two columns each, warps every eighth row
  const uint32_t* bk = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(A.b_k) +
                                                         static_cast<size_t>(h) * d * r) + lane;
  const bool mine = there && 2 * lane < r;
  uint32_t word[k8OpRows];
#pragma unroll
  for (int i = 0; i < k8OpRows; ++i) {
    const int k = warp + k8OpWarps * i;
    word[i] = mine && k < d ? __ldg(bk + k * (r / 2)) : 0u;
  }
  const float q = there && tid < d ? __bfloat162float(static_cast<const __nv_bfloat16*>(
                                         A.q)[(static_cast<size_t>(b) * A.H + h) * d + tid])
                                   : 0.f;
  s_q[tid] = q;
  uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(q) & 0x7fffffffu);
  if (lane == 0) s_max[0][warp] = top;
  __syncthreads();
  float p = 0.f;  // (threads 0 .. r - 1)
  if (r > 0) {
    float a0 = 0.f, a1 = 0.f;
#pragma unroll
    for (int i = 0; i < k8OpRows; ++i) {
      a0 = fmaf(s_q[warp + k8OpWarps * i], bf_lo(word[i]), a0);
      a1 = fmaf(s_q[warp + k8OpWarps * i], bf_hi(word[i]), a1);
    }
    if (mine)
      for (int k = warp + k8OpWarps * k8OpRows; k < d; k += k8OpWarps) {
        const uint32_t w = __ldg(bk + k * (r / 2));
        a0 = fmaf(s_q[k], bf_lo(w), a0);
        a1 = fmaf(s_q[k], bf_hi(w), a1);
      }
    s_part[warp][2 * lane] = a0;
    s_part[warp][2 * lane + 1] = a1;
    __syncthreads();
    if (tid < r) {
#pragma unroll
      for (int i = 0; i < k8OpWarps; ++i) p += s_part[i][tid];
    }
    top = __reduce_max_sync(0xffffffffu, __float_as_uint(p) & 0x7fffffffu);
    if (lane == 0) s_max[1][warp] = top;
    __syncthreads();
    if (tid < r) s_part[0][tid] = p;
    __syncthreads();
  }
  float up[2], down[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    top = 0u;
    if (i == 0 || r > 0)
      for (int k = 0; k < k8OpWarps; ++k) top = max(top, s_max[i][k]);
    const int e = max(static_cast<int>(top >> 23) - 127, -100);
    up[i] = pow2(7 - e);
    // (infinities and NaN make the scores NaN)
    down[i] = e == 128 ? __uint_as_float(0x7fffffffu) : pow2(e - 7) * A.scale_log2;
    if (e == 128) up[i] = 0.f;
  }
  // the parts of this thread's columns: chunk tid / 128 of q, chunks tid / 128 and 2 further of p
  const int col = tid & 127, j0 = tid >> 7;
  uint32_t qv[k8QParts], zv[2][k8Parts];
  auto split = [](float x, auto& v) {
#pragma unroll
    for (uint32_t& y : v) {
      y = e4m3x2(x, 0.f);
      x = (x - from_e4m3x2(y).x) * 16.f;
    }
  };
  split(128 * j0 + col < d ? s_q[128 * j0 + col] * up[0] : 0.f, qv);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = 128 * (j0 + 2 * k) + col - hl * r;  // this head's latent column
    split(c >= 0 && c < r ? s_part[0][c] * up[1] : 0.f, zv[k]);
  }
  const bool empty = there && __ldg(A.seq_lens + b) <= 0;
  pdl_wait();  // the launch before may still read the workspace
  unsigned char* img = A.images + (static_cast<size_t>(b) * A.groups + (h >> 3)) * A.img_bytes;
  if (j0 < A.nd) {
#pragma unroll
    for (int i = 0; i < k8QParts; ++i) {
      const int n = hl * k8QParts + i;
      img[j0 * (k8NQ * 128) + n * 128 + (col ^ ((n & 7) << 4))] = static_cast<unsigned char>(qv[i]);
    }
  }
  img += A.nd * (k8NQ * 128);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = j0 + 2 * k;
    if (j >= A.nz) continue;
#pragma unroll
    for (int i = 0; i < k8Parts; ++i) {
      const int n = hl * k8Parts + i;
      img[j * (k8N * 128) + n * 128 + (col ^ ((n & 7) << 4))] = static_cast<unsigned char>(zv[k][i]);
    }
  }
  img += A.nz * (k8N * 128);
  if (tid < 2) reinterpret_cast<float*>(img)[8 * tid + hl] = there ? down[tid] : 0.f;
  if (hl == 0 && tid == 0) A.arrived[b * A.groups + (h >> 3)] = 0;
  if (h == 0 && b == 0 && tid == 0) *A.status = 0u;
  if (empty) {  // nothing to attend
    if (tid < d) A.out[(static_cast<size_t>(b) * A.H + h) * d + tid] = 0.f;
    if (tid == 0 && A.lse) A.lse[static_cast<size_t>(b) * A.H + h] = -INFINITY;
  }
}

// ================================================================== the scan
// (112 registers a thread at most: the next call's operand CTAs then fit beside a scan CTA.  With 115, 8 x 4096 rows
// took 18.6 us a call for 16.5.)
__global__ void __launch_bounds__(k8Threads, 1)
    lrkv_decode8_kernel(const __grid_constant__ Maps8 M, const __grid_constant__ Args8 A) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  // full/empty: ring slots; ifull/iempty: operands; sfull/sempty: scores; pfull: probabilities; pv: their
  // products done (and the probabilities' buffer free); oempty: a chunk's products read; mdone: every MMA done;
  // mlfirst: the first piece's maxima and denominators written
  __shared__ uint64_t full[k8MaxSlots], empty[k8MaxSlots], ifull[2], iempty[2], sfull[2], sempty[2], pfull[2], pv[2],
      oempty[k8MaxD + k8MaxZ], mdone, mlfirst;
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail, s_bad, s_images, s_copies[2];  // copies issued
  // the first sequence's first CTA, pieces (0: another CTA joins them) and number; the last one's
  __shared__ int s_first[3], s_last[3];
  // [tile parity][half][warp]: maxima of 4 scores, largest and smallest value scale of the shared rows, of the latents;
  // [half][warp]: maxima of 4 + 4 products
  __shared__ __align__(16) float s_red[2][2][4][8], s_top[2][4][8];
  __shared__ float s_fac[4][24];                      // [tile % 4]: alpha[8], factors of the products: latents[8], shared[8]
  __shared__ float s_sum[2][4][4];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  volatile int* fail = &s_fail;

  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int B = A.B, H = A.H, r = A.r, group = blockIdx.y, h0 = group * k8Heads;
  const int heads = min(k8Heads, H - h0);
  const int nd = A.nd, nz = (heads * r + 127) / 128;
  int* pre = reinterpret_cast<int*>(smem);

  // ---- barriers, TMEM, sequence starts in tiles -----------------------------
  if (tid == 0) {
    for (int i = 0; i < k8MaxSlots; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 1 + k8Softmax);
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], k8Softmax);
      mbar_init(&pfull[i], k8Softmax);
      mbar_init(&pv[i], 1);
    }
    for (int i = 0; i < k8MaxD + k8MaxZ; ++i) mbar_init(&oempty[i], k8Values);
    mbar_init(&mdone, 2);
    mbar_init(&mlfirst, 2);
    s_fail = s_bad = s_images = s_copies[0] = s_copies[1] = 0;
    s_first[1] = s_last[1] = 0;
    fence_barrier_init();
  }
  if (warp == 13) tmem_alloc(&tmem_base, k8Cols);
  int bad = 0;
  for (int b = tid; b < B; b += k8Threads) {
    int L = A.seq_lens[b];
    if (L < 0 || L > A.max_len) {
      bad = 1;
      L = min(max(L, 0), A.max_len);
    }
    pre[b + 1] = L / k8Rows + (L % k8Rows != 0);
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
  const int G = max(1, min(static_cast<int>(gridDim.x), N));
  const int c = blockIdx.x;
  const bool work = N > 0 && c < G;
  const int g0 = work ? static_cast<int>(static_cast<long long>(c) * N / G) : 0;
  const int g1 = work ? static_cast<int>(static_cast<long long>(c + 1) * N / G) : 0;
  auto cta_of = [&](int tile) -> int {  // (N G < 2^32 but for absurd CTA counts)
    if (static_cast<unsigned long long>(N) * G >> 32) return cta_of_token(tile, N, G);
    return static_cast<int>(((tile + 1u) * G - 1u) / static_cast<uint32_t>(N));
  };
  auto rows_of = [&](int b) { return min(max(__ldg(A.seq_lens + b), 0), A.max_len); };

  TileWalk w;
  if (!work) {
    // nothing to do
  } else if (warp < k8Softmax) {
    // ---- softmax: row 32 quad + lane of a tile, heads 4 half .. + 3 of the group ----------
    const int quad = warp & 3, half = warp >> 2, row = 32 * quad + lane, hb = h0 + 4 * half;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    const bool vec = H % 4 == 0;
    float m[4], l[4], fq[4], fz[4];
    int cur_b = -1, L = 0, i = 0, piece = -1;
    // scales of this thread's row: shared key and value, latents' keys and values
    float nks = 0.f, nvs = 0.f, nkz[4], nvz[4];
    auto load_scales = [&](const TileWalk& t) {
      const int row_b = k8Rows * t.t0 + row;
      nks = nvs = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) nkz[k] = nvz[k] = 0.f;
      if (row_b >= rows_of(t.b)) return;
      size_t blk = static_cast<size_t>(t.b) * A.blocks + row_b / kBlock8;
      if (A.block_table) {
        const int page = __ldg(A.block_table + static_cast<size_t>(t.b) * A.max_blocks + (row_b >> A.page_shift));
        if (page < 0 || page >= A.num_pages) return;
        blk = static_cast<size_t>(page) * A.blocks + (row_b & ((1 << A.page_shift) - 1)) / kBlock8;
      }
      nks = __ldg(A.cache.k_s_scale + blk);
      nvs = __ldg(A.cache.v_s_scale + blk);
      if (r == 0) return;
      const float* kz = A.cache.z_k_scale + blk * H + hb;
      const float* vz = A.cache.z_v_scale + blk * H + hb;
      if (vec && hb < H) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(kz)), e = __ldg(reinterpret_cast<const float4*>(vz));
        nkz[0] = a.x; nkz[1] = a.y; nkz[2] = a.z; nkz[3] = a.w;
        nvz[0] = e.x; nvz[1] = e.y; nvz[2] = e.z; nvz[3] = e.w;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (hb + k < H) {
            nkz[k] = __ldg(kz + k);
            nvz[k] = __ldg(vz + k);
          }
      }
    };
    bool more = walk_first(w, pre, B, g0, g1);
    if (more) load_scales(w);
    pdl_wait();  // the launch before may still read the workspace
    for (; more; ++i) {
      TileWalk nx = w;
      const bool nmore = walk_next(nx, pre, B, g1, 1);
      const bool last = !nmore || nx.b != w.b;
      if (w.b != cur_b) {
        cur_b = w.b;
        ++piece;
        L = rows_of(w.b);
        wait8_warp(&ifull[piece & 1], static_cast<uint32_t>(piece >> 1) & 1u, fail, A.wait_limit);
        const float* f = reinterpret_cast<const float*>(smem + A.off_img + (piece & 1) * A.img_pad + A.img_bytes - 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          fq[k] = f[4 * half + k];
          fz[k] = f[8 + 4 * half + k];
          m[k] = -INFINITY;
          l[k] = 0.f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&iempty[piece & 1]);
      }
      const int rows = min(k8Rows, L - k8Rows * w.t0);
      float ks = nks, vs = nvs, kz[4], vz[4], zmax = 0.f, zmin = INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        kz[k] = nkz[k];
        vz[k] = nvz[k];
        if (row < rows && r > 0 && hb + k < H) {
          zmax = fmaxf(zmax, vz[k]);
          zmin = fminf(zmin, vz[k]);
        }
      }
      zmax = warp_max(zmax);
      zmin = warp_min(zmin);
      float smax = warp_max(row < rows ? vs : 0.f), smin = warp_min(row < rows ? vs : INFINITY);
      if (nmore) load_scales(nx);

      // the scores
      uint32_t dq[16], dz[24];
      wait8_warp(&sfull[i & 1], static_cast<uint32_t>(i >> 1) & 1u, fail, A.wait_limit);
      tc_fence_after();
      const uint32_t sb = at + k8S + (i & 1) * k8SWidth;
      tmem_ld<16>(sb + 16 * half, dq);
      if (r > 0) {
        tmem_ld<16>(sb + k8NQ + 24 * half, dz);
        tmem_ld<8>(sb + k8NQ + 24 * half + 16, dz + 16);
      } else {
#pragma unroll
        for (int k = 0; k < 24; ++k) dz[k] = 0u;
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&sempty[i & 1]);
      float s[4], top[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = join<4>(dq + 4 * k) * (fq[k] * ks), y = join<6>(dz + 6 * k) * (fz[k] * kz[k]);
        s[k] = row < rows ? x + y : -INFINITY;
        top[k] = warp_max(s[k]);
      }
      // maxima over the tile
      float(*red)[8] = s_red[i & 1][half];
      if (lane == 0) {
        *reinterpret_cast<float4*>(&red[quad][0]) = make_float4(top[0], top[1], top[2], top[3]);
        *reinterpret_cast<float4*>(&red[quad][4]) = make_float4(smax, smin, zmax, zmin);
      }
      bar_named(1 + half, 128);
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const float4 a = *reinterpret_cast<const float4*>(&red[o][0]), e = *reinterpret_cast<const float4*>(&red[o][4]);
        top[0] = fmaxf(top[0], a.x); top[1] = fmaxf(top[1], a.y);
        top[2] = fmaxf(top[2], a.z); top[3] = fmaxf(top[3], a.w);
        smax = fmaxf(smax, e.x); smin = fminf(smin, e.y);
        zmax = fmaxf(zmax, e.z); zmin = fminf(zmin, e.w);
      }
      // one online softmax per head: the sum over the tiles before's maximum, probabilities over the tile's own
      float xs[4], xz[4], ps[4], pz[4], alpha[4], beta[4], below = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        top[k] = fmaxf(top[k], -0x1.fffffep127f);  // (a tile of scores that are -inf: no weight)
        const float mx = fmaxf(m[k], top[k]), p = row < rows ? exp2f(s[k] - top[k]) : 0.f;
        alpha[k] = m[k] == -INFINITY ? 0.f : exp2f(m[k] - mx);
        beta[k] = exp2f(top[k] - mx);
        below = fminf(below, top[k] - mx);
        m[k] = mx;
        l[k] = fmaf(l[k], alpha[k], p * beta[k]);
        xs[k] = xz[k] = p;
      }
      // The probabilities times their block's value scale, over powers of two (of the shared values, of the latents)
      // that bring the tile's largest product of a head to between 2 and 256.  Scales within 2^6 of one another: over
      // the power in the largest scale.
      if (smax <= 64.f * smin && zmax <= 64.f * zmin && fmaxf(smax, zmax) < 0x1p100f && fminf(smin, zmin) > 0x1p-100f &&
          below > -64.f) {
        const float us = vs * (down_to_one(smax) * 128.f), uz = zmax > 0.f ? down_to_one(zmax) * 128.f : 0.f;
        const float fs = power_in(smax) * (1.f / 128.f), fz = power_in(zmax) * (1.f / 128.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          xs[k] *= us;
          xz[k] *= vz[k] * uz;
          ps[k] = fs * beta[k];
          pz[k] = fz * beta[k];
        }
      } else {
        // Any scales, as m 2^e: over a power of two 2^E next to the largest 2^(x + e), x = log2 of the probability,
        // found in a turn of its own.  The probability, which may be too small for a number, does not enter by itself.  (E
        // from -119 on: a 2^-30th of 2^-126 is no number any more.  All tiles this way: 19.5 us for 8 x 4096 rows, 16
        // heads, rank 28, d_h 64, for 17.2; with the turn taken along with that of the scores: 17.7.)
        float es, ez[4];
        const float ms = split_scale(vs, es) * 128.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          vz[k] = split_scale(vz[k], ez[k]) * 128.f;
          s[k] -= m[k];
          ps[k] = warp_max(s[k] + es);
          pz[k] = warp_max(s[k] + ez[k]);
        }
        if (lane == 0) {
          *reinterpret_cast<float4*>(&s_top[half][quad][0]) = make_float4(ps[0], ps[1], ps[2], ps[3]);
          *reinterpret_cast<float4*>(&s_top[half][quad][4]) = make_float4(pz[0], pz[1], pz[2], pz[3]);
        }
        bar_named(1 + half, 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ps[k] = pz[k] = -119.f;
#pragma unroll
          for (int o = 0; o < 4; ++o) {  // (NaN is left out)
            ps[k] = fmaxf(ps[k], ceilf(s_top[half][o][k]));
            pz[k] = fmaxf(pz[k], ceilf(s_top[half][o][4 + k]));
          }
          xs[k] = ms * exp2_ftz(s[k] + (es - ps[k]));
          xz[k] = vz[k] * exp2_ftz(s[k] + (ez[k] - pz[k]));
          ps[k] = pow2(static_cast<int>(ps[k]) - 7);
          pz[k] = pow2(static_cast<int>(pz[k]) - 7);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row >= rows) xs[k] = xz[k] = 0.f;
      // into the operand of the value products, once the ones before are done with it
      if (i > 1) wait8_warp(&pv[i & 1], static_cast<uint32_t>((i >> 1) - 1) & 1u, fail, A.wait_limit);
      unsigned char* to = smem + A.off_p + (i & 1) * (2 * k8PBytes) + (row >> 3) * k8PRows + (row & 7) * 16;
      if (quad == 0 && lane == 0) {
        float* fac = s_fac[i & 3];  // (tile i - 4 is read: the products of i - 2 waited for those of i - 3 to be)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          fac[4 * half + k] = alpha[k];
          fac[8 + 4 * half + k] = pz[k];
          fac[16 + 4 * half + k] = ps[k];
        }
      }
      auto put = [&](float* x, unsigned char* p) {
        uint32_t v[k8Parts];
#pragma unroll
        for (int t = 0; t < k8Parts; ++t) {
          const uint32_t lo = e4m3x2(x[0], x[1]), hi = e4m3x2(x[2], x[3]);
          v[t] = lo | hi << 16;
          if (t + 1 < k8Parts) {
            const float2 a = from_e4m3x2(lo), e = from_e4m3x2(hi);
            x[0] = (x[0] - a.x) * 16.f;
            x[1] = (x[1] - a.y) * 16.f;
            x[2] = (x[2] - e.x) * 16.f;
            x[3] = (x[3] - e.y) * 16.f;
          }
        }
        *reinterpret_cast<uint4*>(p + half * k8PGroup) = make_uint4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint2*>(p + 2 * k8PGroup + 8 * half) = make_uint2(v[4], v[5]);
      };
      put(xs, to);
      if (r > 0) put(xz, to + k8PBytes);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&pfull[i & 1]);
      if (last) {  // the piece's maxima and denominators
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);
          if (lane == 0) s_sum[half][quad][k] = l[k];
        }
        bar_named(1 + half, 128);
        if (quad == 0 && lane < 4 && hb + lane < H) {
          float* pml = A.part_ml + (static_cast<size_t>(w.b + c) * H + hb + lane) * 2;
          pml[0] = lane == 0 ? m[0] : lane == 1 ? m[1] : lane == 2 ? m[2] : m[3];
          pml[1] = (s_sum[half][0][lane] + s_sum[half][1][lane]) + (s_sum[half][2][lane] + s_sum[half][3][lane]);
          if (piece == 0) __threadfence();
        }
        __syncwarp();
        if (piece == 0 && quad == 0 && lane == 0) mbar_arrive_cta(&mlfirst);
        bar_named(1 + half, 128);
      }
      w = nx;
      more = nmore;
    }
  } else if (warp < k8Softmax + k8Values) {
    // ---- value sums: column 32 quad + lane of every chunk ------------------------------
    const int quad = warp & 3, col = 32 * quad + lane, d = A.dh;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    float os[k8MaxD][k8Heads], oz[k8MaxZ];
    int head[k8MaxZ], lo[k8MaxZ], hi[k8MaxZ];  // this column's head; the warp's first and last
#pragma unroll
    for (int j = 0; j < k8MaxZ; ++j) {
      head[j] = lo[j] = -1;
      hi[j] = -2;
      if (j < nz) {
        head[j] = (128 * j + col) / r;
        lo[j] = (128 * j + 32 * quad) / r;
        hi[j] = min((128 * j + 32 * quad + 31) / r, heads - 1);
      }
    }
    auto let_go = [&](int chunk) {  // a chunk's products are read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&oempty[chunk]);
    };
    pdl_wait();  // the launch before may still read the workspace
    int i = 0, cur_b = -1;
    for (bool more = walk_first(w, pre, B, g0, g1); more; ++i) {
      TileWalk nx = w;
      const bool nmore = walk_next(nx, pre, B, g1, 1);
      const bool last = !nmore || nx.b != w.b;
      if (w.b != cur_b) {
        cur_b = w.b;
#pragma unroll
        for (int j = 0; j < k8MaxD; ++j)
#pragma unroll
          for (int k = 0; k < k8Heads; ++k) os[j][k] = 0.f;
#pragma unroll
        for (int j = 0; j < k8MaxZ; ++j) oz[j] = 0.f;
      }
      wait8_warp(&pv[i & 1], static_cast<uint32_t>(i >> 1) & 1u, fail, A.wait_limit);
      tc_fence_after();
      const float* fac = s_fac[i & 3];
#pragma unroll
      for (int j = 0; j < k8MaxD; ++j) {
        if (j >= nd) break;
        uint32_t v[k8N];
        tmem_ld<16>(at + k8Os + j * k8N, v);
        tmem_ld<16>(at + k8Os + j * k8N + 16, v + 16);
        tmem_ld<16>(at + k8Os + j * k8N + 32, v + 32);
        tmem_wait_ld();
        let_go(j);
#pragma unroll
        for (int k = 0; k < k8Heads; ++k)
          os[j][k] = fmaf(os[j][k], fac[k], join_values(v + 16 * (k >> 2), v + 32 + 8 * (k >> 2), k & 3) * fac[16 + k]);
      }
#pragma unroll
      for (int j = 0; j < k8MaxZ; ++j) {
        if (j >= nz) break;
        for (int q = lo[j] >> 2; q <= hi[j] >> 2; ++q) {  // four heads at a time (the same for the whole warp)
          uint32_t v[16], u[8];
          tmem_ld<16>(at + k8Oz + j * k8N + 16 * q, v);
          tmem_ld<8>(at + k8Oz + j * k8N + 32 + 8 * q, u);
          tmem_wait_ld();
          float x = join_values(v, u, 0);
#pragma unroll
          for (int k = 1; k < 4; ++k) {
            const float y = join_values(v, u, k);
            if ((head[j] & 3) == k) x = y;
          }
          if (head[j] >> 2 == q) oz[j] = fmaf(oz[j], fac[head[j]], x * fac[8 + head[j]]);
        }
        let_go(nd + j);
      }
      if (last) {
        float* out = A.part_acc + (static_cast<size_t>(w.b + c) * H + h0) * (d + r);
#pragma unroll
        for (int j = 0; j < k8MaxD; ++j) {
          if (j < nd && 128 * j + col < d) {
#pragma unroll
            for (int k = 0; k < k8Heads; ++k)
              if (k < heads) out[static_cast<size_t>(k) * (d + r) + 128 * j + col] = os[j][k];
          }
        }
#pragma unroll
        for (int j = 0; j < k8MaxZ; ++j)
          if (j < nz && head[j] < heads)
            out[static_cast<size_t>(head[j]) * (d + r) + d + 128 * j + col - head[j] * r] = oz[j];
        if (nmore && pre[w.b] < g0) {  // the first of several: this CTA is done with it
          __threadfence();
          bar_named(5, 32 * k8Values);
          if (warp == k8Softmax && lane == 0) {
            wait8(&mlfirst, 0u, fail, A.wait_limit);
            __threadfence();
            const int c0 = cta_of(pre[w.b]), n = c - c0 + 1;
            s_first[0] = c0;
            s_first[1] = atomicAdd(&A.arrived[w.b * A.groups + group], 1) == n - 1 ? n : 0;
            __threadfence();
          }
          __syncwarp();
        }
      }
      w = nx;
      more = nmore;
    }
  } else if (warp == 12 || warp == 15) {
    // ---- copies of the keys (warp 12, with each piece's operands) and of the values (15), a
    // ring each: with one ring for both, a parity could not tell a phase from the one two
    // before it when one side runs ahead.  A lane per box; a slot is let go by the MMAs that
    // read it, so its last copy has landed -----------------------------------------------
    const bool values = warp == 15, leader = elect();
    const int slots = A.slots[values], s0 = values ? A.slots[0] : 0, nc = nd + nz;
    int copies = 0, piece = 0;
    bool ok = true, first = true;
    Place8 at8;
    Pieces8 w8 = {};
    auto operands = [&](int b) {
      ok = ok && (piece < 2 || wait8_warp(&iempty[piece & 1], static_cast<uint32_t>((piece >> 1) - 1) & 1u, fail,
                                          A.wait_limit));
      if (ok && leader) {
        mbar_arrive_expect_tx(&ifull[piece & 1], A.img_bytes);
        tma_load_1d(smem + A.off_img + (piece & 1) * A.img_pad,
                    A.images + (static_cast<size_t>(b) * A.groups + group) * A.img_bytes, A.img_bytes,
                    &ifull[piece & 1]);
        s_images = piece + 1;
      }
      ++piece;
    };
    auto begin = [&] {  // the first operands are the launch before's
      first = false;
      pdl_wait();
      operands(w8.b);
    };
    for (bool more = w8.first(pre, B, g0, g1); more && ok; more = w8.next(pre, B, g1)) {
      const int L = uniform(rows_of(w8.b));
      if (!values && !first) operands(w8.b);
      for (int t = w8.t0; t < w8.t0 + w8.n && ok; ++t) {
        const int padded = round_up(min(k8Rows, L - k8Rows * t), k8Step);
        const bool tail = padded < k8Rows;
        const int box = tail ? A.tail_box : A.box, boxes = padded / box;
        const int at = k8Rows * t + lane * box;  // this lane's first row
        int y = at, z = w8.b;
        if (A.block_table && lane < boxes) {
          y = at & ((1 << A.page_shift) - 1);
          z = A.num_pages;  // rows past the sequence, or whose page is not one of the pool's: zeros
          if (at < L) {
            const int page = __ldg(A.block_table + static_cast<size_t>(w8.b) * A.max_blocks + (at >> A.page_shift));
            if (page >= 0 && page < A.num_pages) z = page; else s_bad = 1;
          }
        }
        const CUtensorMap* map = &M.map[(tail ? 4 : 0) + (values ? 1 : 0)];
        int x = 0;
        for (int j = 0; j < nc; ++j, x += 128, at8.move(1, slots)) {
          if (j == nd) {
            x = h0 * r;
            map += 2;
          }
          const int slot = s0 + at8.slot;
          // (with the ring full the first scores are waited for)
          if (first && !values && copies == slots) begin();
          if (copies >= slots) ok = ok && wait8_warp(&empty[slot], at8.phase ^ 1u, fail, A.wait_limit);
          if (!ok) break;
          ++copies;
          if (leader) {
            mbar_arrive_expect_tx(&full[slot], padded * 128);
            s_copies[values] = copies;
          }
          __syncwarp();
          if (lane < boxes)
            tma_load_3d(smem + A.off_ring + slot * k8Box + lane * box * 128, map, x, y, z, &full[slot]);
        }
        if (first && !values) begin();
        first = false;
      }
    }
  } else if (warp == 13) {
    // ---- scores of a tile: q against the shared rows, p against the latents -----------------
    const bool leader = elect();
    const uint32_t td = uniform(tmem);
    const uint64_t ring = smem_desc(smem_u32(smem + A.off_ring), 16, 1024, 2);
    const uint64_t img = smem_desc(smem_u32(smem + A.off_img), 16, 1024, 2);
    Place8 at8;
    Pieces8 w8 = {};
    int i = 0, piece = 0;
    bool ok = true;
    for (bool more = w8.first(pre, B, g0, g1); more && ok; more = w8.next(pre, B, g1), ++piece) {
      ok = wait8_warp(&ifull[piece & 1], static_cast<uint32_t>(piece >> 1) & 1u, fail, A.wait_limit);
      for (int t = 0; t < w8.n && ok; ++t, ++i) {
        const int a = i & 1;
        ok = i < 2 || wait8_warp(&sempty[a], static_cast<uint32_t>((i >> 1) - 1) & 1u, fail, A.wait_limit);
        const uint32_t sd = td + k8S + a * k8SWidth;
        uint64_t bd = img + static_cast<uint32_t>((piece & 1) * (A.img_pad / 16));
        for (int j = 0; j < nd + nz && ok; ++j, at8.move(1, A.slots[0])) {
          ok = wait8_warp(&full[at8.slot], at8.phase, fail, A.wait_limit);
          if (!ok) break;
          tc_fence_after();
          const bool z = j >= nd;
          const int left = z ? heads * r - 128 * (j - nd) : A.dh - 128 * j;
          if (leader) {
            mma8_box(sd + (z ? k8NQ : 0), ring + static_cast<uint32_t>(at8.slot * (k8Box / 16)), 2, bd, 2,
                     z ? idesc8(k8N, 0) : idesc8(k8NQ, 0), min(4, (left + 31) >> 5), z ? j == nd : j == 0);
            tc_commit(&empty[at8.slot]);
          }
          __syncwarp();
          bd += (z ? k8N : k8NQ) * 8;
        }
        if (ok && leader) {
          tc_commit(&sfull[a]);
          if (t + 1 == w8.n) tc_commit(&iempty[piece & 1]);
        }
        __syncwarp();
      }
    }
    if (leader) tc_commit(&mdone);  // every MMA of this warp, also of a pass that gave up
  } else if (warp == 14) {
    // ---- values of a tile: columns x rows of the boxes against the probabilities ------------
    const bool leader = elect();
    const uint32_t td = uniform(tmem);
    const uint64_t ring = smem_desc(smem_u32(smem + A.off_ring + A.slots[0] * k8Box), 16, 1024, 2);
    const uint64_t pd = smem_desc(smem_u32(smem + A.off_p), k8PRows, k8PGroup, 0);
    Place8 at8;
    Pieces8 w8 = {};
    int i = 0;
    bool ok = true;
    for (bool more = w8.first(pre, B, g0, g1); more && ok; more = w8.next(pre, B, g1)) {
      const int L = uniform(rows_of(w8.b));
      for (int t = w8.t0; t < w8.t0 + w8.n && ok; ++t, ++i) {
        const int rows = min(k8Rows, L - k8Rows * t), steps = (rows + k8Step - 1) / k8Step;
        ok = wait8_warp(&pfull[i & 1], static_cast<uint32_t>(i >> 1) & 1u, fail, A.wait_limit);
        for (int j = 0; j < nd + nz && ok; ++j, at8.move(1, A.slots[1])) {
          const int slot = A.slots[0] + at8.slot;
          ok = wait8_warp(&full[slot], at8.phase, fail, A.wait_limit) &&
               (i == 0 || wait8_warp(&oempty[j], static_cast<uint32_t>(i - 1) & 1u, fail, A.wait_limit));
          if (!ok) break;
          if (rows < steps * k8Step) {
            // rows past the sequence (which may hold anything) must not meet their zero probabilities as 0 x NaN
            uint4* past = reinterpret_cast<uint4*>(smem + A.off_ring + slot * k8Box + rows * 128);
            for (int k = lane; k < 8 * (steps * k8Step - rows); k += 32) past[k] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          const bool z = j >= nd;
          if (leader) {
            mma8_box(td + (z ? k8Oz + (j - nd) * k8N : k8Os + j * k8N),
                     ring + static_cast<uint32_t>(at8.slot * (k8Box / 16)), 256,
                     pd + ((i & 1) * 2 + (z ? 1 : 0)) * (k8PBytes / 16), 4 * k8PRows / 16, idesc8(k8N, 1), steps,
                     true);
            tc_commit(&empty[slot]);
          }
          __syncwarp();
        }
        if (ok && leader) tc_commit(&pv[i & 1]);
        __syncwarp();
      }
    }
    if (leader) tc_commit(&mdone);
  }

  // ---- the end.  A sequence's pieces are joined by the last CTA done with one of them: in their
  // order, with the latents' sum lifted through B_h^V.  A CTA has said so already of its first
  // sequence if that one ends inside its range (above), says so now of its last one, and joins
  // alone what lies between.  The group's B_h^V, the same for all of them, is on its way to shared
  // memory before it is known who joins ------------------------------------------------------
  pdl_wait();
  int last_n = 0;
  if (tid == 32 && work) {
    TileWalk e;
    walk_first(e, pre, B, g0, g1);
    s_first[2] = e.b;
    walk_first(e, pre, B, g1 - 1, g1);
    const int c0 = pre[e.b] < g0 ? cta_of(pre[e.b]) : c, c1 = pre[e.b + 1] > g1 ? cta_of(pre[e.b + 1] - 1) : c;
    last_n = c1 - c0 + 1;
    s_last[2] = e.b;
    s_last[0] = c0;
  }
  if (warp < k8Softmax + k8Values) __threadfence();  // the last piece's results, for the CTA that joins it
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int W = A.dh + r, d = A.dh;
  // [lift][d] rows of B_h^V, over the operands, the probabilities and the ring: a row every odd number of 16 bytes,
  // so that the threads of a warp, a row each, read different banks
  unsigned char* s_b = smem + A.off_img;
  const int pitch = A.pitch, vec = A.vec, parts = r / vec;  // columns of a copy, copies of a row
  auto fetch_b = [&](int k0) {  // (all warps but warp 1, which finds out meanwhile who joins)
    const int t = tid - (warp > 1 ? 32 : 0), threads = k8Threads - 32;
    if (warp == 1 || parts == 0) return;
    const int rows = threads / parts, part = t % parts;  // (r <= 64: at least 15 rows at once)
    int row = t / parts;
    if (row >= rows) return;
    const __nv_bfloat16* src =
        static_cast<const __nv_bfloat16*>(A.b_v) + (static_cast<size_t>(h0 + k0) * d + row) * r + part * vec;
    uint32_t dst = smem_u32(s_b) + static_cast<uint32_t>(row * pitch + part * vec * 2);
    for (; row < min(A.lift, heads - k0) * d; row += rows, src += rows * r, dst += rows * pitch) {
      if (vec == 8)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      else if (vec == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
    }
  };
  // (a pass that did not give up has waited for every copy and every product)
  const bool gave_up = *fail;
  if (work && !gave_up) fetch_b(0);
  if (warp == 13) {
    if (work && !mbar_wait_bounded(&mdone, 0u) && lane == 0) record_status(A.status, kDevTimeout);
    __syncwarp();
    tmem_dealloc(tmem, k8Cols);
  } else if (tid == 0) {
    if (gave_up) {
      for (int v = 0, s0 = 0; v < 2; s0 += A.slots[v], ++v)
        for (int i = max(0, s_copies[v] - A.slots[v]); i < s_copies[v]; ++i)
          mbar_wait_bounded(&full[s0 + i % A.slots[v]], static_cast<uint32_t>(i / A.slots[v]) & 1u);
      for (int i = max(0, s_images - 2); i < s_images; ++i)
        mbar_wait_bounded(&ifull[i & 1], static_cast<uint32_t>(i >> 1) & 1u);
    }
    const uint32_t bits = (bad || s_bad ? kDevBounds : 0u) | (gave_up ? kDevTimeout : 0u);
    if (bits) record_status(A.status, bits);
  } else if (tid == 32 && work) {
    int n = last_n;
    if (n > 1 && atomicAdd(&A.arrived[s_last[2] * A.groups + group], 1) != n - 1) n = 0;
    __threadfence();
    s_last[1] = n;
  }
  __syncthreads();
  if (!work || gave_up) return;
  const int pad = round_up(W, 4);
  float* s_w = reinterpret_cast<float*>(s_b + A.lift * d * pitch);  // [8][pieces] weights, then [8][pad] sums
  const int b_first = s_first[2], b_last = s_last[2];
  const size_t step = static_cast<size_t>(H) * W;
  constexpr int kCols = 2, kDeep = 10;  // pairs of columns a thread sums at once, pieces it has under way
  struct Joined {  // a sequence to join, and what its first pieces hold
    int b, c0, n;
    float2 ml, v[kCols][kDeep];
  } x;
  auto fetch = [&](Joined& x, int e0, int i0) {
    const float* acc = A.part_acc + (static_cast<size_t>(x.b + x.c0) * H + h0) * W;
#pragma unroll
    for (int j = 0; j < kCols; ++j)
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int e = 2 * (e0 + tid + j * k8Threads);
        x.v[j][i] = i0 + i < x.n && e < heads * W ? __ldcg(reinterpret_cast<const float2*>(acc + (i0 + i) * step + e))
                                                  : make_float2(0.f, 0.f);
      }
  };
  auto piece = [&](const Joined& x, int i) {  // its maximum and denominator for head `warp`
    const float2* ml = reinterpret_cast<const float2*>(A.part_ml) + static_cast<size_t>(x.b + x.c0) * H + h0 + warp;
    return i < x.n && warp < heads ? __ldcg(ml + static_cast<size_t>(i) * H) : make_float2(-INFINITY, 0.f);
  };
  auto find = [&](Joined& x) {  // the first one to join from x.b on
    for (; x.b <= b_last; ++x.b) {
      x.n = pre[x.b + 1] > pre[x.b] ? 1 : 0;
      x.c0 = c;
      if (x.b == b_last) {
        x.n = s_last[1];
        x.c0 = s_last[0];
      } else if (x.b == b_first && pre[x.b] < g0) {
        x.n = s_first[1];
        x.c0 = s_first[0];
      }
      if (x.n == 0) continue;
      x.ml = piece(x, lane);
      fetch(x, 0, 0);
      return true;
    }
    return false;
  };
  x.b = b_first;
  bool have_b = true;
  for (bool any = find(x); any;) {
    const int b = x.b, n = x.n;
    float* s_o = s_w + k8Heads * n;
    if (warp < heads) {
      float m = x.ml.x;
      for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, piece(x, i).x);
      m = warp_max(m);
      auto weight = [&](float of) { return of == -INFINITY ? 0.f : exp2f(of - m); };
      const float own = weight(x.ml.x);
      float l = own * x.ml.y;
      for (int i = lane + 32; i < n; i += 32) {
        const float2 ml = piece(x, i);
        l = fmaf(weight(ml.x), ml.y, l);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const float inv = 1.f / l;
      if (lane < n) s_w[warp * n + lane] = own * inv;
      for (int i = lane + 32; i < n; i += 32) s_w[warp * n + i] = weight(piece(x, i).x) * inv;
      if (lane == 0 && A.lse) A.lse[static_cast<size_t>(b) * H + h0 + warp] = (m + log2f(l)) * kLn2;
    }
    for (int e0 = 0; 2 * e0 < heads * W; e0 += kCols * k8Threads) {  // (W is even: a pair is of one head)
      int k[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) k[j] = min(2 * (e0 + tid + j * k8Threads) / W, heads - 1);
      if (e0 == 0) __syncthreads();  // (the weights)
      float2 y[kCols] = {};
      for (int i0 = 0; i0 < n; i0 += kDeep) {
        if (e0 > 0 || i0 > 0) fetch(x, e0, i0);
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
          for (int i = 0; i < kDeep; ++i)
            if (i0 + i < n) {
              y[j].x = fmaf(s_w[k[j] * n + i0 + i], x.v[j][i].x, y[j].x);
              y[j].y = fmaf(s_w[k[j] * n + i0 + i], x.v[j][i].y, y[j].y);
            }
      }
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int e = 2 * (e0 + tid + j * k8Threads);
        if (e < heads * W) *reinterpret_cast<float2*>(s_o + k[j] * (pad - W) + e) = y[j];
      }
    }
    ++x.b;
    any = find(x);  // the next one's loads are under way during this one's lift
    float* out = A.out + (static_cast<size_t>(b) * H + h0) * d;
    for (int k0 = 0; k0 < heads; k0 += A.lift) {
      if (!have_b) fetch_b(k0);
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
      for (int e = tid; e < min(A.lift, heads - k0) * d; e += k8Threads) {
        const int k = k0 + e / d;
        const float* o = s_o + k * pad;
        const unsigned char* row = s_b + e * pitch;
        float y[4] = {o[e - (k - k0) * d], 0.f, 0.f, 0.f};
        int i = 0;
#pragma unroll 1
        for (; i + 8 <= r; i += 8) {
          const uint4 a = *reinterpret_cast<const uint4*>(row + 2 * i);
          const float4 z = *reinterpret_cast<const float4*>(o + d + i);
          const float4 zz = *reinterpret_cast<const float4*>(o + d + i + 4);
          y[0] = fmaf(bf_hi(a.x), z.y, fmaf(bf_lo(a.x), z.x, y[0]));
          y[1] = fmaf(bf_hi(a.y), z.w, fmaf(bf_lo(a.y), z.z, y[1]));
          y[2] = fmaf(bf_hi(a.z), zz.y, fmaf(bf_lo(a.z), zz.x, y[2]));
          y[3] = fmaf(bf_hi(a.w), zz.w, fmaf(bf_lo(a.w), zz.z, y[3]));
        }
        for (; i < r; i += 2) {
          const uint32_t a = *reinterpret_cast<const uint32_t*>(row + 2 * i);
          y[1] = fmaf(bf_hi(a), o[d + i + 1], fmaf(bf_lo(a), o[d + i], y[1]));
        }
        out[k0 * d + e] = (y[0] + y[1]) + (y[2] + y[3]);
      }
      have_b = A.lift >= heads;  // (it stays for the next sequence)
      __syncthreads();
    }
  }
}

// ======================================================================= host
namespace {

lrkv_status decode8_check(const lrkv_dims* d) {
  const lrkv_status st = cache8_check_dims(d);
  if (st != LRKV_OK) return st;
  return d->dtype == LRKV_BF16 ? LRKV_OK : LRKV_ERR_UNSUPPORTED;
}

// Carves the workspace up from `ws` on; returns its size.
size_t decode8_bind(Args8& A, void* ws) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    unsigned char* p = static_cast<unsigned char*>(ws) + off;
    off += (bytes + 255) / 256 * 256;
    return ws ? p : nullptr;
  };
  const size_t slots = static_cast<size_t>(A.B + A.grid) * A.H;
  A.status = reinterpret_cast<uint32_t*>(take(256));
  A.arrived = reinterpret_cast<int*>(take(sizeof(int) * A.B * A.groups));
  A.part_ml = reinterpret_cast<float*>(take(sizeof(float) * slots * 2));
  A.part_acc = reinterpret_cast<float*>(take(sizeof(float) * slots * (A.dh + A.r)));
  A.images = take(static_cast<size_t>(A.B) * A.groups * A.img_bytes);
  return off;
}

// Shared memory of the join: B_h^V of `lift` heads, weights of the pieces, sums.
long long decode8_lift_bytes(const Args8& A, int lift) {
  return 1ll * lift * A.dh * A.pitch + 4ll * k8Heads * (A.grid + round_up(A.dh + A.r, 4));
}

lrkv_status decode8_plan(const lrkv_dims& d, int num_sms, Args8& A, size_t* bytes) {
  std::memset(&A, 0, sizeof(A));
  A.B = d.batch; A.H = d.heads; A.dh = d.head_dim; A.r = d.rank; A.max_len = d.max_len;
  const float scale = d.scale > 0.f ? d.scale : 1.f / std::sqrt(static_cast<float>(d.head_dim));
  A.scale_log2 = scale * kLog2e;
  A.wait_limit = wait_limit_cycles();
  A.groups = (A.H + k8Heads - 1) / k8Heads;
  A.nd = (A.dh + 127) / 128;
  A.nz = (std::min(A.H, k8Heads) * A.r + 127) / 128;
  A.grid = std::min(std::max(1, num_sms / A.groups), 1024);  // (the join keeps a weight per piece in shared memory)
  A.img_bytes = A.nd * k8NQ * 128 + A.nz * k8N * 128 + 128;
  A.img_pad = round_up(A.img_bytes, 1024);
  int off = round_up((A.B + 1) * 4, 1024);
  A.off_img = off; off += 2 * A.img_pad;
  A.off_p = off; off += 4 * k8PBytes;
  A.off_ring = off;
  const int budget = 224 * 1024;  // (3 KB of the 227 for the static part and the alignment)
  const int slots = std::min(k8MaxSlots, (budget - off) / k8Box);
  if (slots < 4) return LRKV_ERR_UNSUPPORTED;
  A.slots[0] = slots / 2;
  A.slots[1] = slots - A.slots[0];
  A.smem_bytes = off + slots * k8Box + 1024;
  A.pitch = (round_up(2 * A.r, 16) / 16 | 1) * 16;
  const long long room = off + slots * k8Box - A.off_img;
  for (A.lift = k8Heads; A.lift > 1 && decode8_lift_bytes(A, A.lift) > room;) A.lift /= 2;
  if (decode8_lift_bytes(A, A.lift) > room) return LRKV_ERR_UNSUPPORTED;
  *bytes = decode8_bind(A, nullptr);
  return LRKV_OK;
}

}  // namespace

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_decode8_workspace_size(const lrkv_dims* dims, size_t* bytes) {
  if (!bytes) return LRKV_ERR_INVALID_ARG;
  const lrkv_status st = lrkv::decode8_check(dims);
  if (st != LRKV_OK) return st;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  lrkv::Args8 A;
  return lrkv::decode8_plan(*dims, sms, A, bytes);
}

lrkv_status lrkv_decode8(const lrkv_dims* dims, const void* q, int page_size, int num_pages,
                         const int32_t* block_table, const lrkv_cache8* cache, const void* b_k, const void* b_v,
                         const int32_t* seq_lens, float* out, float* lse, void* ws, size_t ws_bytes,
                         lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_decode8");
  lrkv_status st = lrkv::decode8_check(dims);
  if (st != LRKV_OK) return st;
  if ((st = lrkv::cache8_check(dims, cache)) != LRKV_OK) return st;
  if (!q || !seq_lens || !out || (dims->rank > 0 && (!b_k || !b_v))) return LRKV_ERR_INVALID_ARG;
  if (!lrkv::cache8_a16(q) || reinterpret_cast<uintptr_t>(b_k) % 4 != 0 || reinterpret_cast<uintptr_t>(b_v) % 4 != 0)
    return LRKV_ERR_INVALID_ARG;
  if ((st = lrkv::cache8_check_paging(dims, page_size, num_pages, block_table)) != LRKV_OK) return st;
  if (!ws) return LRKV_ERR_WORKSPACE;
  if (!lrkv::cache8_a16(ws)) return LRKV_ERR_INVALID_ARG;
  const int sms = lrkv::device_sm_count();
  if (sms < 1) return LRKV_ERR_CUDA;
  lrkv::Args8 A;
  size_t need = 0;
  if ((st = lrkv::decode8_plan(*dims, sms, A, &need)) != LRKV_OK) return st;
  if (ws_bytes < need) return LRKV_ERR_WORKSPACE;
  lrkv::decode8_bind(A, ws);
  A.cache = *cache;
  A.q = q; A.b_k = b_k; A.b_v = b_v;
  A.seq_lens = seq_lens; A.out = out; A.lse = lse;
  int rows = A.max_len, lead = A.B;
  if (block_table) {
    A.block_table = block_table;
    A.max_blocks = A.max_len / page_size;
    A.num_pages = num_pages;
    while ((1 << A.page_shift) < page_size) ++A.page_shift;
    rows = page_size;
    lead = num_pages;
  }
  A.blocks = (rows + lrkv::kBlock8 - 1) / lrkv::kBlock8;
  A.box = block_table ? std::min(page_size, lrkv::k8Rows) : lrkv::k8Rows;
  A.tail_box = std::min(A.box, lrkv::k8Step);
  const uintptr_t bv = reinterpret_cast<uintptr_t>(b_v);
  A.vec = A.r % 8 == 0 && bv % 16 == 0 ? 8 : A.r % 4 == 0 && bv % 8 == 0 ? 4 : 2;
  lrkv::Maps8 M;
  std::memset(&M, 0, sizeof(M));
  const void* const held[4] = {cache->k_s, cache->v_s, cache->z_k, cache->z_v};
  for (int i = 0; i < 8; ++i)
    if ((i & 2) == 0 || A.r > 0) {
      const int width = (i & 2) == 0 ? A.dh : A.H * A.r;
      if (!lrkv::make_tmap_3d_u8(&M.map[i], held[i & 3], width, rows, lead, 128, i < 4 ? A.box : A.tail_box))
        return LRKV_ERR_CUDA;
    }
  const void* kern = reinterpret_cast<const void*>(lrkv::lrkv_decode8_kernel);
  if (lrkv::ensure_kernel_smem(kern, A.smem_bytes, true) != cudaSuccess) return LRKV_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(A.groups * lrkv::k8Heads, A.B);
  cfg.blockDim = dim3(lrkv::k8OpThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, lrkv::lrkv_decode8_operands_kernel, A) != cudaSuccess) return LRKV_ERR_CUDA;
  cfg.gridDim = dim3(A.grid, A.groups);
  cfg.blockDim = dim3(lrkv::k8Threads);
  cfg.dynamicSmemBytes = A.smem_bytes;
  return cudaLaunchKernelEx(&cfg, lrkv::lrkv_decode8_kernel, M, A) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

}  // extern "C"
