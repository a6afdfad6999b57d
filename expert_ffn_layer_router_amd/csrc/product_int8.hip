// LDS-tiled products of 8-bit codes, with the scales of rows and columns.
#include "product_core.h"

namespace moe {

void launch_product_int8(const ProductArgs& a, const ProductPlan& p, Result res, hipStream_t s) {
  if (res == Result::kGated)
    launch_tiles<Num::kInt8, Pass::kForward, Result::kGated>(a, p, s);
  else if (res == Result::kWide)
    launch_tiles<Num::kInt8, Pass::kForward, Result::kWide>(a, p, s);
  else
    launch_tiles<Num::kInt8, Pass::kForward, Result::kHalf>(a, p, s);
}

}  // namespace moe
