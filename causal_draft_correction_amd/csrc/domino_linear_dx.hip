// Products of linear layers: the gradient of x: dpre w (the weights lie across k).
#define DH_NT 256
#define DH_NS dhl
#include "dh_gemm.h"

namespace DH_NS {

hipError_t product_dx(const Gemm &g, int shape, hipStream_t st) { return launch_gemm<true, false>(g, shape, st); }

}  // namespace DH_NS
