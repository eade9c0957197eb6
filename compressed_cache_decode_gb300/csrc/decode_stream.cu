// decode_stream.cu — plan, tensor maps and launch of the bf16 split-KV scan
// (decode_stream_kernel.cuh), with the scan's plain instantiations; the ones
// that also leave the scores are compiled in decode_stream_weighted.cu.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>

#include "decode_stream_kernel.cuh"
#include "tmap.h"

namespace lrkv {

StreamFn stream_fn_weighted(const DecodePlan& P);  // decode_stream_weighted.cu

namespace {

StreamFn stream_fn(const DecodePlan& P) { return P.scores ? stream_fn_weighted(P) : pick_stream<false>(P); }

}  // namespace

// Fills the streaming-kernel fields of an already sized plan.
static lrkv_status stream_plan_impl(DecodePlan& P);

lrkv_status stream_plan(DecodePlan& P_out) {
  DecodePlan P = P_out;
  const lrkv_status st = stream_plan_impl(P);
  if (st == LRKV_OK) P_out = P;
  return st;
}

static lrkv_status stream_plan_impl(DecodePlan& P) {
  const int dh = P.dh, r = P.r, H = P.H;
  if (!(dh == 64 || dh == 128)) return LRKV_ERR_UNSUPPORTED;
  if (r % 4 != 0 || r > 64) return LRKV_ERR_UNSUPPORTED;
  P.stream = 1;
  P.T = kT;
  P.Hp = round_up(H, 16);
  P.mt = P.Hp / 16;
  P.grid = std::max(1, P.grid / P.mt);
  P.ngw = kPairs;  // one partial per warp pair and piece
  P.nthreads = kThreadsS;
  P.span = 128;
  P.box_cols = 64;
  P.nbox = dh / 64;
  P.kv_bytes = round_up(kT * dh * 2, 1024);
  if (r > 0) {
    // latent segment: hs heads (a power of two dividing H) whose hs r
    // latents are a multiple of 16 elements and fit a box with 8 spare
    P.hs = 0;
    for (int hs = 16; hs >= 1; hs >>= 1)
      if (H % hs == 0 && (hs * r) % 16 == 0 && hs * r + 8 <= 256) { P.hs = hs; break; }
    if (P.hs == 0) return LRKV_ERR_UNSUPPORTED;
    P.segw = P.hs * r;
    P.segp = P.segw + 8;  // (segw / 8) is even, so segp / 8 is odd
    P.nsb = 16 / P.hs;
    P.zt_bytes = P.nsb * kT * P.segp * 2;
    P.kst = r / 2;  // 16-wide steps over the 8 r latents of 8 heads
    if (P.kst > 32) return LRKV_ERR_UNSUPPORTED;
    // shared offset of step n of half h2: latent column j = 8 h2 r + 16 n
    for (int h2 = 0; h2 < 2; ++h2)
      for (int n = 0; n < 32; ++n) {
        const int j = 8 * h2 * r + 16 * std::min(n, P.kst - 1);
        P.zo[h2][n] = (j / P.segw) * kT * P.segp * 2 + (j % P.segw) * 2;
      }
  } else {
    P.hs = 1; P.segw = 0; P.segp = 0; P.nsb = 0; P.zt_bytes = 0; P.kst = 0;
    for (int h2 = 0; h2 < 2; ++h2)
      for (int n = 0; n < 32; ++n) P.zo[h2][n] = 0;
  }
  P.pq_bytes = round_up(16 * dh * 2 + 16 * r * (P.weighted ? 6 : 4), 128);
  // absorb roles: 16 heads x r/4 column groups x bk_dsplit head-dim parts
  P.bk_dsplit = 1;
  while (r > 0 && 16 * (r / 4) * P.bk_dsplit * 2 <= kThreadsS && P.bk_dsplit * 2 <= dh / 4) P.bk_dsplit *= 2;
  P.bk_warps = r > 0 ? (16 * (r / 4) * P.bk_dsplit + 31) / 32 : 1;
  P.stage_bytes = round_up(2 * P.kv_bytes + 2 * P.zt_bytes, 1024);
  // the key-scale slot (post-projection RMSNorm decode) when the stages
  // still fit as many of it (set below)
  P.off_ks = 2 * P.kv_bytes + 2 * P.zt_bytes;  // 256-byte aligned
  P.ks_bytes = 0;
  P.ks_tma = 0;
  const int pf_bytes = 2 * (dh / 16) * 32 * 8;  // q fragments of both halves

  // shared memory: barriers | prefix | p/q buffers | q fragments | ring
  auto layout = [&](int stages) {
    int off = kHeaderBytes;  // barriers, stage records, step offsets, tile cursors
    P.off_prefix = off; off = round_up(off + (P.B + 1) * 4, 128);
    P.off_pq = off; off = round_up(off + 2 * P.pq_bytes, 128);
    P.off_pf = off; off = round_up(off + std::max(pf_bytes, 16), 1024);
    P.off_kv = off; off += stages * P.stage_bytes;
    return off + 1024;  // alignment slack
  };
  const int budget = 226 * 1024;  // opt-in limit (227 KB) less static shared memory
  const char* cap_env = std::getenv("LRKV_DECODE_STREAM_STAGES");  // tuning: at most this many stages
  const int cap = (cap_env && *cap_env) ? std::max(2, std::atoi(cap_env)) : 16;
  int stages = 0;
  while (stages < std::min(16, cap) && layout(stages + 1) <= budget) ++stages;
  if (stages < 2) return LRKV_ERR_UNSUPPORTED;
  P.stages = stages;
  {
    const int plain = P.stage_bytes;
    P.stage_bytes = round_up(P.off_ks + 16 * kKsBoxT * 4, 1024);
    if (layout(P.stages) <= budget)
      P.ks_bytes = 16 * kKsBoxT * 4;
    else
      P.stage_bytes = plain;
  }
  P.smem_bytes = layout(P.stages);
  // B^K of a row tile staged through the last ring stages when it fits
  // (leaving at least one stage for the first tiles), those stages getting
  // their tiles after the absorb; otherwise each absorb thread loads its
  // columns at entry.  Tuning: LRKV_DECODE_BK_REGS=1 takes the register
  // path whenever a thread's columns are one chunk (d_h / bk_dsplit <=
  // kBkChunk rows); measured slower on 8 x 4K rows of 16 heads, rank 28:
  // the absorb from registers took ~5.5K cycles against ~2.4K from shared
  // memory.
  {
    P.bk_head_bytes = dh * r * 2;
    const long long bk_bytes = 16ll * P.bk_head_bytes;
    const int nbk = r > 0 ? static_cast<int>((bk_bytes + P.stage_bytes - 1) / P.stage_bytes) : 0;
    const char* regs_env = std::getenv("LRKV_DECODE_BK_REGS");
    const bool one_chunk = dh / P.bk_dsplit <= kBkChunk && regs_env && regs_env[0] == '1';
    P.bk_stages = (r > 0 && nbk < stages && !one_chunk) ? nbk : 0;
  }
  P.pfw = 0;  // L2 prefetch window beyond the ring (tiles); set with the grid
  return stream_fn(P) ? LRKV_OK : LRKV_ERR_UNSUPPORTED;
}

// Host preparation of a streaming launch: the latent tensor maps and the
// kernel's shared-memory attribute (set once per kernel and size).
lrkv_status stream_prepare(const DecodePlan& P, CUtensorMap* tm_zk, CUtensorMap* tm_zv, CUtensorMap* tm_ks) {
  const StreamFn kern = stream_fn(P);
  if (!kern) return LRKV_ERR_UNSUPPORTED;
  std::memset(tm_zk, 0, sizeof(*tm_zk));
  std::memset(tm_zv, 0, sizeof(*tm_zv));
  std::memset(tm_ks, 0, sizeof(*tm_ks));
  // key scales [B][H][max_len] fp32 in boxes of [16 heads][kKsBoxT rows]
  if (P.ks_tma &&
      !make_tmap_3d_f32(tm_ks, P.key_scale, static_cast<uint64_t>(P.max_len), static_cast<uint64_t>(P.H),
                        static_cast<uint64_t>(P.B), kKsBoxT, 16u))
    return LRKV_ERR_CUDA;
  if (P.r > 0) {
    // z[b][t][h][c] viewed as [b][segment][t][hs r]: dims (inner first)
    // {hs r, rows, H / hs, sequences}, strides t: H r, segment: hs r, b: rows H r
    // (rows, sequences) = (max_len, B), or (page_size, pages) for a paged cache
    const uint64_t row = static_cast<uint64_t>(P.H) * P.r * 2;
    const uint64_t dims[4] = {static_cast<uint64_t>(P.segw), static_cast<uint64_t>(P.map_len),
                              static_cast<uint64_t>(P.H / P.hs), static_cast<uint64_t>(P.map_seqs)};
    const uint64_t strides[3] = {row, static_cast<uint64_t>(P.segw) * 2, row * P.map_len};
    const uint32_t box[4] = {static_cast<uint32_t>(P.segp), static_cast<uint32_t>(kT),
                             static_cast<uint32_t>(P.nsb), 1u};
    if (!make_tmap_4d_bf16_strided(tm_zk, P.z_k, dims, strides, box) ||
        !make_tmap_4d_bf16_strided(tm_zv, P.z_v, dims, strides, box))
      return LRKV_ERR_CUDA;
  }
  // the largest size set so far per kernel (per device: the attribute is a
  // property of the function in the current context)
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, int> set_bytes;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LRKV_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  int& have = set_bytes[{dev, reinterpret_cast<const void*>(kern)}];
  if (have < P.smem_bytes) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P.smem_bytes) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
      return LRKV_ERR_CUDA;
    have = P.smem_bytes;
  }
  return LRKV_OK;
}

lrkv_status stream_launch(const DecodePlan& P, cudaStream_t stream, bool pdl, const CUtensorMap& tm_k,
                          const CUtensorMap& tm_v, const CUtensorMap& tm_zk, const CUtensorMap& tm_zv,
                          const CUtensorMap& tm_ks) {
  const StreamFn kern = stream_fn(P);
  if (!kern) return LRKV_ERR_UNSUPPORTED;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(P.grid, P.mt);
  cfg.blockDim = dim3(P.nthreads);
  cfg.dynamicSmemBytes = P.smem_bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, P, tm_k, tm_v, tm_zk, tm_zv, tm_ks) == cudaSuccess ? LRKV_OK : LRKV_ERR_CUDA;
}

}  // namespace lrkv
