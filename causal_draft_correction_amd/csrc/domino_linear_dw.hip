// Products of linear layers: the gradient of w: dpre^T x (both operands lie across k).
#define DH_NT 256
#define DH_NS dhl
#include "dh_gemm.h"

namespace DH_NS {

hipError_t product_dw(const Gemm &g, int shape, hipStream_t st) { return launch_gemm<true, true>(g, shape, st); }

}  // namespace DH_NS
