// Gradients of rows: dz [rows][n] times weights [n][k], whose adjacent elements are output columns.
#include "ffn_gemm.h"

namespace ffn {

int run_dx(Product& p, const Tiling& t, int dtype, hipStream_t stream) {
  return with_type16(dtype, [&](auto type) {
    return launch_product<decltype(type), kInside, kOutsideK, false>(p, t, stream);
  });
}

}  // namespace ffn
