// Kernels of the gated linear recurrence: the adjoint, backward in time (recur_core.cuh).
#include "recur_core.cuh"

namespace sla {

sla_status recur_backward(int32_t dtype, int32_t gate, const void *args, void *work, cudaStream_t s)
{
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        return run_recur<S, true>(gate, *(const RecurArgs<S> *)args, work, s);
    });
}

}  // namespace sla
