// LDS-tiled gradients of the 16-bit products: with respect to the rows (the
// contraction runs over w's rows) and to the weights (over the group's rows).
#include "product_core.h"

namespace moe {

template <Num T>
static void launch_grad(const ProductArgs& a, const ProductPlan& p, Pass pass, Result res, hipStream_t s) {
  if (pass == Pass::kInputGrad)
    launch_tiles<T, Pass::kInputGrad, Result::kHalf>(a, p, s);
  else if (res == Result::kWide)
    launch_tiles<T, Pass::kWeightGrad, Result::kWide>(a, p, s);
  else
    launch_tiles<T, Pass::kWeightGrad, Result::kHalf>(a, p, s);
}

void launch_product_grad(const ProductArgs& a, const ProductPlan& p, Num num, Pass pass, Result res, hipStream_t s) {
  if (num == Num::kFp16)
    launch_grad<Num::kFp16>(a, p, pass, res, s);
  else
    launch_grad<Num::kBf16>(a, p, pass, res, s);
}

}  // namespace moe
