// decode_stream_weighted.cu — the scan's instantiations that also leave the
// scores (lrkv_decode_weighted), in a translation unit of their own so that
// the two sets compile side by side.
#include "decode_stream_kernel.cuh"

namespace lrkv {

StreamFn stream_fn_weighted(const DecodePlan& P) { return pick_stream<true>(P); }

}  // namespace lrkv
