// Gradient products: of the inputs (the weight strided along the sum) and of the weights (both
// operands strided along the sum).
#include "dense_gemm.h"

namespace moe {

moe_status dense_nn_product(const DenseProduct &p, const DensePlan &pl, const EpiStore &e, float *part, const DenseSide &side,
                            DenseLater *later, hipStream_t s) {
    return dense_run<kFormNN>(p, pl, e, part, s, side, later);
}
moe_status dense_tn_product(const DenseProduct &p, const DensePlan &pl, const EpiStore &e, float *part, const DenseSide &side,
                            const DenseLater &later, hipStream_t s) {
    return dense_run<kFormTN>(p, pl, e, part, s, side, nullptr, later);
}

}  // namespace moe
