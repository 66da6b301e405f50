// Products of linear layers: x w^T (both operands lie along k).
#define DH_NT 256
#define DH_NS dhl
#include "dh_gemm.h"

namespace DH_NS {

hipError_t product_y(const Gemm &g, int shape, hipStream_t st) { return launch_gemm<false, false>(g, shape, st); }

}  // namespace DH_NS
