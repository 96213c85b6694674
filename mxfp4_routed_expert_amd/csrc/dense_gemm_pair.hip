// Gate and up products of one tile in one kernel, with the activation or its gradient in the epilogue.
#include "dense_gemm.h"

namespace moe {

moe_status dense_gate_product(const DenseProduct &p, const DensePlan &pl, const EpiGate &e, float *part, hipStream_t s) {
    return dense_run<kFormNT>(p, pl, e, part, s);
}
moe_status dense_gate_bwd_product(const DenseProduct &p, const DensePlan &pl, const EpiGateBwd &e, float *part,
                                  hipStream_t s) {
    return dense_run<kFormNT>(p, pl, e, part, s);
}

}  // namespace moe
