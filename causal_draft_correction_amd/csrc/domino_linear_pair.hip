// Products of linear layers: the gradients of x and w in one launch, for layers so small that launches count.
#define DH_NT 256
#define DH_NS dhl
#include "dh_gemm.h"

namespace DH_NS {

// Blocks [0, n) take the tiles of x's gradient, those from n on those of w's (64 x 64 both).
template <typename TW, typename TX, typename TG>
__global__ __launch_bounds__(256, 2) void k_gemm_pair(Gemm x, Gemm w, int n)
{
    typedef Tile<TW, TG, true, false, 64, 64, 32, 32, STEP_K<TW, TG>> X;
    typedef Tile<TX, TG, true, true, 64, 64, 32, 32, STEP_K<TX, TG>> W;
    __shared__ uint4 lds[X::LDS_ALL > W::LDS_ALL ? X::LDS_ALL : W::LDS_ALL];
    const int block = static_cast<int>(blockIdx.x);
    if (block >= n)
        W::run(w, block - n, lds);
    else if (block < x.ti * x.tj * x.splits)
        X::run(x, block, lds);
}

hipError_t product_pair(const Gemm &x, const Gemm &w, hipStream_t st)
{
    const int n = (x.ti * x.tj * x.splits + 7) / 8 * 8;  // (so that the second product's blocks begin on the first die)
    const dim3 grid(static_cast<unsigned>(n + w.ti * w.tj * w.splits));
    const auto launch = [&](auto tw, auto tx, auto tg) {
        hipLaunchKernelGGL((k_gemm_pair<decltype(tw), decltype(tx), decltype(tg)>), grid, dim3(256), 0, st, x, w, n);
    };
    const auto by_g = [&](auto tw, auto tx) { x.b.f32 ? launch(tw, tx, float{}) : launch(tw, tx, bf16s{}); };
    const auto by_x = [&](auto tw) { w.a.f32 ? by_g(tw, float{}) : by_g(tw, bf16s{}); };
    x.a.f32 ? by_x(float{}) : by_x(bf16s{});
    return hipGetLastError();
}

}  // namespace DH_NS
