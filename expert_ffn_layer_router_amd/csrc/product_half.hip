// LDS-tiled products of 16-bit rows and weights, forward.
#include "product_core.h"

namespace moe {

template <Num T>
static void launch_half(const ProductArgs& a, const ProductPlan& p, Result res, hipStream_t s) {
  if (res == Result::kGated)
    launch_tiles<T, Pass::kForward, Result::kGated>(a, p, s);
  else
    launch_tiles<T, Pass::kForward, Result::kHalf>(a, p, s);
}

void launch_product_half(const ProductArgs& a, const ProductPlan& p, Num num, Result res, hipStream_t s) {
  if (num == Num::kFp16)
    launch_half<Num::kFp16>(a, p, res, s);
  else
    launch_half<Num::kBf16>(a, p, res, s);
}

}  // namespace moe
