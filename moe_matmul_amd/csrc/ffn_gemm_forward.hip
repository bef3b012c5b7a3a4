// Forward products of nvfp4_ffn.h: rows and weights with adjacent k.
#include "ffn_gemm.h"

namespace ffn {

int run_forward(Product& p, const Tiling& t, int dtype, bool gated, hipStream_t stream) {
  return with_type16(dtype, [&](auto type) {
    using T = decltype(type);
    return gated ? launch_product<T, kInside, kInside, true>(p, t, stream)
                 : launch_product<T, kInside, kInside, false>(p, t, stream);
  });
}

}  // namespace ffn
