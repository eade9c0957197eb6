// quantize.cu — rows of the factored cache into its 8-bit form
// (lrkv_quantize): e4m3 numbers with a power-of-two scale for each block of 16
// rows, tensor and head (a shared row counts as one head).
//
// Memory bounds it: every new element is read once (2 or 4 bytes) and written
// once (1 byte).  A CTA takes the keys' or the values' half of one block, a
// thread a few columns of all 16 rows, which stay in registers while the
// largest magnitudes of the block's heads are found in shared memory; so the
// rows are read once, all loads of a thread in flight together.  Maxima do not
// depend on the order in which they are taken: the results are the same every
// time.
//
// A block that was begun before (a decode step, or a prompt that goes on) keeps
// its scale unless the new rows need a larger one; then its earlier rows are
// rounded anew in place.
//
// Measured on GB300, back-to-back calls of a graph: 8 prompts of 4-8K rows, bf16,
// 32 heads of rank 48, d_h 128: 80.3 us, 6.5 TB/s read and written (0.97 of a
// measured copy's 6.7); 32 decode steps, rank 56, in pages: 3.0 us, a launch's
// latency (a caller's own 10 us a call are the bound there).
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "cache8.h"
#include "decode_plan.h"
#include "lrkv.h"
#include "ptx.cuh"
#include "trace.h"

namespace lrkv {

namespace {

constexpr int kQzThreads = 512;  // at most
// Registers a thread: three CTAs of 224 threads an SM (32 heads of rank 48) keep more rows under way than two, and
// four leave a thread too few for its 16 rows (96: 95 us, 80: 81, 72: 92 for 8 prompts of 4-8K rows).
constexpr int kQzRegs = 80;

struct QuantizeArgs {
  int n_new, max_len, H, d, r;
  int slab_heads;                  // heads of a CTA
  int page_shift, num_pages, max_blocks;
  const int32_t* block_table;      // or NULL
  const int32_t* start_pos;
  const int32_t* new_lens;         // or NULL
  const void* rows[4];             // k_s, z_k, v_s, z_v
  unsigned char* cache[4];
  float* scale[4];
  uint32_t* status;                // or NULL
};

// V elements of a row.  peak(): the largest bits of a magnitude, of any kind, or 0x7f800000 and up where one is
// not finite; finite(): of the finite ones.
template <typename T, int V>
struct Vec;
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
template <int V>
struct Vec<__nv_bfloat16, V> {
  uint32_t w[V / 2];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (V == 8) {
      const uint4 u = __ldg(static_cast<const uint4*>(p));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (V == 4) {
      const uint2 u = __ldg(static_cast<const uint2*>(p));
      w[0] = u.x; w[1] = u.y;
    } else {
      w[0] = __ldg(static_cast<const uint32_t*>(p));
    }
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]); }
  // two magnitudes at a time: the bits of bf16 are ordered as integers
  __device__ __forceinline__ void peak(uint32_t& m) const {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  }
  static __device__ __forceinline__ uint32_t peak_of(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  // times a power of two: exact, but for what e4m3 has no bits for
  __device__ __forceinline__ void scaled(float inv, float* y) const {
    const __nv_bfloat162 by = __float2bfloat162_rn(inv);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), by);
      const uint32_t u = *reinterpret_cast<const uint32_t*>(&p);
      y[2 * i] = bf_lo(u);
      y[2 * i + 1] = bf_hi(u);
    }
  }
};
template <int V>
struct Vec<float, V> {
  float f[V];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (V == 4) {
      const float4 u = __ldg(static_cast<const float4*>(p));
      f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
    } else {
      const float2 u = __ldg(static_cast<const float2*>(p));
      f[0] = u.x; f[1] = u.y;
    }
  }
  __device__ __forceinline__ float get(int i) const { return f[i]; }
  __device__ __forceinline__ void peak(uint32_t& m) const {
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  }
  static __device__ __forceinline__ uint32_t peak_of(uint32_t m) { return m; }
  __device__ __forceinline__ void scaled(float inv, float* y) const {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = f[i] * inv;
  }
};
template <int V>
__device__ __forceinline__ void store8(unsigned char* p, const float* x) {
  const uint32_t a = e4m3x2(x[0], x[1]);
  if constexpr (V == 2) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(a);
  } else {
    const uint32_t lo = a | e4m3x2(x[2], x[3]) << 16;
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = lo;
    else *reinterpret_cast<uint2*>(p) = make_uint2(lo, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
  }
}

// y, the fp32 number nearest to y + rest, moved by its last bit towards it where that makes the bit 1: never a tie of
// fewer bits then, so that a second rounding gives what one of y + rest would.
__device__ __forceinline__ float sticky(float y, float rest) {
  const uint32_t u = __float_as_uint(y);
  if ((u & 1u) != 0u || y == 0.f || !(rest != 0.f) || !(fabsf(rest) <= 3e38f)) return y;
  return __uint_as_float((rest > 0.f) == (y > 0.f) ? u + 1u : u - 1u);
}
// The smallest power of two s, 2^-126 at least, with amax <= 448 s = 1.75 * 2^8 s (bits of amax, finite).
__device__ __forceinline__ float scale_for(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 127;  // amax = 1.m * 2^e
  const int k = max((amax & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7, -126);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

}  // namespace

// grid (blocks a sequence's rows can touch, sequences, halves x slabs of heads)
template <typename T, int V>
__global__ void __maxnreg__(kQzRegs) lrkv_quantize_kernel(const __grid_constant__ QuantizeArgs A) {
  extern __shared__ uint32_t s_amax[];  // the shared row, then the slab's heads
  const int b = blockIdx.y, tid = threadIdx.x, half = blockIdx.z & 1, slab = blockIdx.z >> 1;
  pdl_wait();  // the launch before
  const long long start = A.start_pos[b];
  long long n = A.new_lens ? A.new_lens[b] : A.n_new;
  bool bad = n < 0 || n > A.n_new;
  n = min(max(n, 0ll), static_cast<long long>(A.n_new));
  const int first = static_cast<int>(min(max(start, 0ll), static_cast<long long>(A.max_len)));
  const int end = static_cast<int>(min(max(start + n, 0ll), static_cast<long long>(A.max_len)));
  bad = bad || (n > 0 && (start < 0 || start + n > A.max_len));
  if (bad && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) record_status(A.status, kDevBounds);
  // (blocks are compared, not rows: a grid may go on past row 2^31)
  const int block = first / kBlock8 + static_cast<int>(blockIdx.x);
  if (end == 0 || block > (end - 1) / kBlock8) return;
  const int base = block * kBlock8;  // the block's first row
  // where the block lies
  size_t row0 = static_cast<size_t>(b) * A.max_len + base;
  size_t blk = static_cast<size_t>(b) * ((A.max_len + kBlock8 - 1) / kBlock8) + base / kBlock8;
  if (A.block_table) {
    const int page = A.block_table[static_cast<size_t>(b) * A.max_blocks + (base >> A.page_shift)];
    if (page < 0 || page >= A.num_pages) {
      if (blockIdx.z == 0 && tid == 0) record_status(A.status, kDevBounds);
      return;
    }
    row0 = (static_cast<size_t>(page) << A.page_shift) + (base & ((1 << A.page_shift) - 1));
    blk = row0 / kBlock8;
  }
  const int lo = max(first - base, 0), hi = min(end - base, kBlock8);  // the block's new rows
  if (lo >= hi) return;

  // this thread's columns: of the shared row (the first slab's), or of a head
  const int h0 = slab * A.slab_heads, heads = min(A.slab_heads, A.H - h0);
  const int shared = slab == 0 ? A.d / V : 0, per_head = A.r / V;
  const bool mine = tid < shared + heads * per_head, latent = tid >= shared;
  const int head = latent && mine ? (tid - shared) / per_head : 0;
  const int item = latent ? 1 + head : 0, which = 2 * half + (latent ? 1 : 0);
  const int width = latent ? A.H * A.r : A.d;
  const int col = latent ? h0 * A.r + (tid - shared) * V : tid * V;
  const bool owner = mine && (latent ? (tid - shared) % per_head == 0 : tid == 0);
  for (int i = tid; i <= heads; i += blockDim.x) s_amax[i] = 0u;
  Vec<T, V> x[kBlock8];
  const T* src = static_cast<const T*>(A.rows[which]) +
                 (static_cast<long long>(b) * A.n_new + (base - start)) * width + col;
  uint32_t top = 0u;
  if (mine) {
#pragma unroll
    for (int i = 0; i < kBlock8; ++i)
      if (i >= lo && i < hi) x[i].load(src + static_cast<long long>(i) * width);
  }
  float* scale = A.scale[which];
  const size_t at = latent ? blk * A.H + h0 + head : blk;
  const float before = mine && lo > 0 ? scale[at] : 0.f;
  if (mine) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kBlock8; ++i)
      if (i >= lo && i < hi) x[i].peak(m);
    top = Vec<T, V>::peak_of(m);
    if (top >= 0x7f800000u) {  // infinities and NaN do not count
      top = 0u;
#pragma unroll
      for (int i = 0; i < kBlock8; ++i)
        if (i >= lo && i < hi)
#pragma unroll
          for (int k = 0; k < V; ++k) top = max(top, finite_bits(x[i].get(k)));
    }
  }
  __syncthreads();
  if (mine && top) atomicMax(&s_amax[item], top);
  __syncthreads();
  if (!mine) return;
  const float s = fmaxf(before, scale_for(s_amax[item]));
  if (owner) scale[at] = s;
  unsigned char* dst = A.cache[which] + row0 * width + col;
  if ((__float_as_uint(s) & 0x7fffffu) == 0u) {  // a power of two, as all but a caller's own are: x / s is x (1 / s)
    const float inv = 1.f / s;
#pragma unroll
    for (int i = 0; i < kBlock8; ++i)
      if (i >= lo && i < hi) {
        float y[V];
        x[i].scaled(inv, y);
        store8<V>(dst + static_cast<size_t>(i) * width, y);
      }
  } else {  // (the rows once more, one at a time: with this side on `x` the other took 81.5 us for 80.3)
    // (in a range where what the quotient leaves is a number)
    const float up = s < 0x1p-60f ? 0x1p64f : 1.f, d = s * up;
#pragma unroll 1
    for (int i = lo; i < hi; ++i) {
      Vec<T, V> v;
      float y[V];
      v.load(src + static_cast<long long>(i) * width);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float f = v.get(k) * up, p = f / d;
        y[k] = sticky(p, fmaf(-p, d, f));
      }
      store8<V>(dst + static_cast<size_t>(i) * width, y);
    }
  }
  if (lo > 0 && s > before) {  // the earlier rows, to the larger scale
    const float ratio = before / s;  // (exact: s is a power of two)
    for (int i = 0; i < lo; ++i) {
      unsigned char* p = dst + static_cast<size_t>(i) * width;
      float y[V];
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float2 f = from_e4m3x2(*reinterpret_cast<const uint16_t*>(p + k));
        y[k] = f.x * ratio;
        y[k + 1] = f.y * ratio;
        y[k] = sticky(y[k], fmaf(f.x, ratio, -y[k]));
        y[k + 1] = sticky(y[k + 1], fmaf(f.y, ratio, -y[k + 1]));
      }
      store8<V>(p, y);
    }
  }
}

namespace {

using QuantizeFn = void (*)(const QuantizeArgs);

// Columns of a thread: the widest load that no head's columns split.
QuantizeFn quantize_fn(bool bf16, int r, int* v) {
  *v = r % 8 == 0 && bf16 ? 8 : r % 4 == 0 ? 4 : 2;
  if (bf16)
    return *v == 8 ? lrkv_quantize_kernel<__nv_bfloat16, 8>
                   : *v == 4 ? lrkv_quantize_kernel<__nv_bfloat16, 4> : lrkv_quantize_kernel<__nv_bfloat16, 2>;
  return *v == 4 ? lrkv_quantize_kernel<float, 4> : lrkv_quantize_kernel<float, 2>;
}

}  // namespace

}  // namespace lrkv

extern "C" lrkv_status lrkv_quantize(const lrkv_dims* dims, int n_new, const void* k_s, const void* v_s,
                                     const void* z_k, const void* z_v, const int32_t* start_pos,
                                     const int32_t* new_lens, int page_size, int num_pages,
                                     const int32_t* block_table, const lrkv_cache8* cache, void* ws, size_t ws_bytes,
                                     lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_quantize");
  lrkv_status st = lrkv::cache8_check_dims(dims);
  if (st != LRKV_OK) return st;
  if (n_new < 1) return LRKV_ERR_INVALID_ARG;
  if (static_cast<long long>(dims->batch) * n_new > (1LL << 31) - 1) return LRKV_ERR_UNSUPPORTED;
  if ((st = lrkv::cache8_check(dims, cache)) != LRKV_OK) return st;
  if (!k_s || !v_s || !start_pos || (dims->rank > 0 && (!z_k || !z_v))) return LRKV_ERR_INVALID_ARG;
  if (!lrkv::cache8_a16(k_s) || !lrkv::cache8_a16(v_s) ||
      (dims->rank > 0 && (!lrkv::cache8_a16(z_k) || !lrkv::cache8_a16(z_v))))
    return LRKV_ERR_INVALID_ARG;
  if ((st = lrkv::cache8_check_paging(dims, page_size, num_pages, block_table)) != LRKV_OK) return st;
  if (ws && !lrkv::cache8_a16(ws)) return LRKV_ERR_INVALID_ARG;
  if (ws && ws_bytes < 16) return LRKV_ERR_WORKSPACE;
  lrkv::QuantizeArgs A = {};
  A.n_new = n_new; A.max_len = dims->max_len; A.H = dims->heads; A.d = dims->head_dim; A.r = dims->rank;
  A.start_pos = start_pos; A.new_lens = new_lens;
  A.rows[0] = k_s; A.rows[1] = z_k; A.rows[2] = v_s; A.rows[3] = z_v;
  unsigned char* const held[4] = {static_cast<unsigned char*>(cache->k_s), static_cast<unsigned char*>(cache->z_k),
                                  static_cast<unsigned char*>(cache->v_s), static_cast<unsigned char*>(cache->z_v)};
  float* const scales[4] = {cache->k_s_scale, cache->z_k_scale, cache->v_s_scale, cache->z_v_scale};
  std::copy(held, held + 4, A.cache);
  std::copy(scales, scales + 4, A.scale);
  A.status = static_cast<uint32_t*>(ws);
  if (block_table) {
    A.block_table = block_table;
    A.num_pages = num_pages;
    A.max_blocks = dims->max_len / page_size;
    while ((1 << A.page_shift) < page_size) ++A.page_shift;
  }
  int v = 0;
  const lrkv::QuantizeFn kern = lrkv::quantize_fn(dims->dtype == LRKV_BF16, A.r, &v);
  // as many heads a CTA as its threads hold beside a shared row
  const int most = A.r > 0 ? std::max(1, (lrkv::kQzThreads - A.d / v) / (A.r / v)) : A.H;
  const int slabs = A.r > 0 ? (A.H + most - 1) / most : 1;
  A.slab_heads = A.r > 0 ? (A.H + slabs - 1) / slabs : 0;
  const int threads = (A.d / v + A.slab_heads * (A.r / v) + 31) / 32 * 32;
  const long long blocks = std::min<long long>((static_cast<long long>(n_new) + lrkv::kBlock8 - 2) / lrkv::kBlock8 + 1,
                                               (dims->max_len + lrkv::kBlock8 - 1) / lrkv::kBlock8);
  // (launched ahead of the end of the launch before, for which it waits: 83.0 -> 80.5 us for 8 prompts back to back,
  // 3.2 -> 3.0 for 32 single rows in a graph)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), dims->batch, 2 * slabs);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (A.slab_heads + 1) * sizeof(uint32_t);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return cudaLaunchKernelEx(&cfg, kern, A) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}
