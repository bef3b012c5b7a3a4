// Gradients of weights: dz [rows][n] and x [rows][k], summed over an expert's rows.
#include "ffn_gemm.h"

namespace ffn {

int run_dw(Product& p, const Tiling& t, int dtype, hipStream_t stream) {
  return with_type16(dtype, [&](auto type) {
    return launch_product<decltype(type), kOutsideK, kOutsideK, false>(p, t, stream);
  });
}

}  // namespace ffn
