// Forward products (both operands contiguous along the sum) with the linear layer's epilogues.
#include "dense_gemm.h"

namespace moe {

moe_status dense_linear_product(const DenseProduct &p, const DensePlan &pl, const EpiLinear &e, float *part,
                                hipStream_t s) {
    return dense_run<kFormNT>(p, pl, e, part, s);
}
moe_status dense_linear_bwd_product(const DenseProduct &p, const DensePlan &pl, const EpiLinearBwd &e, float *part,
                                    hipStream_t s) {
    return dense_run<kFormNT>(p, pl, e, part, s);
}

}  // namespace moe
