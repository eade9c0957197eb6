// rope_rotate.cu — rotary positions with several axes, applied to the rows of
// a tensor (lrkv_rope_rotate): the queries that lrkv_decode_rope and
// lrkv_decode_rope_axes take already rotated.
//
// Pair k of a head, (x_2k, x_2k+1), belongs to one axis (time, height, width,
// ...): the pairs are cut into consecutive sections, one per axis.  With the
// token's position p on that axis it turns by p theta_k, theta_k = base^(-2k /
// d_h), read from the rotation table (row p, pair k).  One read and one write
// of x bounds it; the turn is fp32 and rounded once.
//
// A thread owns 16 bytes of a head's row (4 pairs of bf16, 2 of fp32) for
// every n-th head of one token, so its cos and sin come from the table once
// per token and stay in registers across the heads.
//
// Four heads' pieces are loaded at once, before the position: one after another
// (a store may alias the next load, so none is hoisted) the long case below ran
// at 4.1 TB/s.
//
// Measured: 2 x 4096 tokens of 32 heads, d_h 128, bf16, three axes (134 MB read
// and written, 20.1 us at the copy rate) 24.6 us, 5.5 TB/s; one token of 32
// sequences 9-11 us a call, which is the launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "decode_plan.h"
#include "host_cache.h"
#include "lrkv.h"
#include "ptx.cuh"
#include "rope_axes.h"
#include "trace.h"

namespace lrkv {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotHeads = 4;  // heads a thread has under way

struct RotateParams {
  long long tokens;        // batch * n
  int H, dh;
  int cols;                // 16-byte pieces of a head's row
  int hpp;                 // heads of one pass of a token
  int tpc;                 // tokens of a CTA
  int max_pos;
  RopeAxes ax;
  const int32_t* positions;  // [tokens][axes]
  const float* table;        // [max_pos][dh]
  const unsigned char* x;
  unsigned char* out;
  uint32_t* status;
};

}  // namespace

template <bool BF16>
__global__ void __launch_bounds__(kRotThreads) lrkv_rope_rotate_kernel(const RotateParams P) {
  constexpr int NP = BF16 ? 4 : 2;  // pairs of a 16-byte piece
  const int col = threadIdx.x % P.cols, group = threadIdx.x / P.cols;
  const long long token = static_cast<long long>(blockIdx.x) * P.tpc + group / P.hpp;
  if (group >= P.tpc * P.hpp || token >= P.tokens) return;
  const size_t head = static_cast<size_t>(P.cols) * 16;
  const size_t base = static_cast<size_t>(token) * P.H * head + static_cast<size_t>(col) * 16;
  // out may be x: every piece is read before the thread that owns it writes it,
  // the first ones before the position and its table entries are waited for
  uint4 v[kRotHeads];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kRotHeads; ++i)
      if (h0 + i * P.hpp < P.H) v[i] = *reinterpret_cast<const uint4*>(P.x + base + (h0 + i * P.hpp) * head);
  };
  int h0 = group % P.hpp;
  load(h0);
  float2 cs[NP];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < NP; ++u) {
    const int k = col * NP + u;
    int p = P.positions[token * P.ax.n + P.ax.axis(k)];
    if (p < 0 || p >= P.max_pos) {
      bad = true;
      p = min(max(p, 0), P.max_pos - 1);
    }
    cs[u] = *reinterpret_cast<const float2*>(P.table + static_cast<size_t>(p) * P.dh + 2 * k);
  }
  if (bad && P.status) atomicOr(P.status, kDevBounds);
  while (true) {
#pragma unroll
    for (int i = 0; i < kRotHeads; ++i) {
      if (h0 + i * P.hpp >= P.H) break;
      const uint32_t in[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        const float a = BF16 ? bf_lo(in[u]) : __uint_as_float(in[2 * u & 3]);
        const float c = BF16 ? bf_hi(in[u]) : __uint_as_float(in[(2 * u + 1) & 3]);
        const float ra = fmaf(a, cs[u].x, -c * cs[u].y), rc = fmaf(a, cs[u].y, c * cs[u].x);
        if (BF16) {
          const __nv_bfloat162 w = __floats2bfloat162_rn(ra, rc);
          o[u] = *reinterpret_cast<const uint32_t*>(&w);
        } else {
          o[2 * u & 3] = __float_as_uint(ra);
          o[(2 * u + 1) & 3] = __float_as_uint(rc);
        }
      }
      *reinterpret_cast<uint4*>(P.out + base + (h0 + i * P.hpp) * head) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    h0 += kRotHeads * P.hpp;
    if (h0 >= P.H) break;
    load(h0);
  }
}

}  // namespace lrkv

extern "C" {

lrkv_status lrkv_rope_rotate(const lrkv_dims* dims, int n, const void* x, const int32_t* positions, int axes,
                             const int* sections, const float* cos_sin, int max_pos, void* out, void* ws,
                             size_t ws_bytes, lrkv_stream_t stream) {
  LRKV_TRACE_CALL("lrkv_rope_rotate");
  using namespace lrkv;
  if (!dims || dims->batch < 1 || dims->heads < 1 || dims->head_dim < 2 || n < 1 || max_pos < 1)
    return LRKV_ERR_INVALID_ARG;
  if (dims->dtype != LRKV_F32 && dims->dtype != LRKV_BF16) return LRKV_ERR_INVALID_ARG;
  if (!x || !positions || !cos_sin || !out) return LRKV_ERR_INVALID_ARG;
  RotateParams P;
  std::memset(&P, 0, sizeof(P));
  if (!rope_axes_make(axes, sections, dims->head_dim, P.ax)) return LRKV_ERR_INVALID_ARG;
  const int esz = dims->dtype == LRKV_BF16 ? 2 : 4;
  if (static_cast<long long>(dims->head_dim) * esz % 16 != 0 || dims->head_dim > 1024) return LRKV_ERR_UNSUPPORTED;
  auto aligned = [](const void* p, unsigned m) { return (reinterpret_cast<uintptr_t>(p) & (m - 1)) == 0; };
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(cos_sin, 8)) return LRKV_ERR_INVALID_ARG;
  if (ws && ws_bytes < 16) return LRKV_ERR_WORKSPACE;
  if (ws && !aligned(ws, 16)) return LRKV_ERR_INVALID_ARG;
  P.tokens = static_cast<long long>(dims->batch) * n;
  P.H = dims->heads; P.dh = dims->head_dim;
  P.cols = dims->head_dim * esz / 16;
  const int groups = kRotThreads / P.cols;
  // heads side by side: as many as leave each thread its kRotHeads
  P.hpp = std::min((P.H + kRotHeads - 1) / kRotHeads, groups);
  P.tpc = std::max(1, groups / P.hpp);
  P.max_pos = max_pos;
  P.positions = positions; P.table = cos_sin;
  P.x = static_cast<const unsigned char*>(x); P.out = static_cast<unsigned char*>(out);
  P.status = static_cast<uint32_t*>(ws);
  const long long blocks = (P.tokens + P.tpc - 1) / P.tpc;
  if (blocks > 0x7fffffffLL) return LRKV_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->dtype == LRKV_BF16)
    lrkv_rope_rotate_kernel<true><<<static_cast<unsigned>(blocks), kRotThreads, 0, s>>>(P);
  else
    lrkv_rope_rotate_kernel<false><<<static_cast<unsigned>(blocks), kRotThreads, 0, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

}  // extern "C"
