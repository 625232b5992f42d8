// router_dense.cuh -- the dense router products (router_gemm.cu) as their
// entry points (router_dense.cu) call them; arguments already checked.
#pragma once

#include "common.cuh"

namespace moe {

size_t router_logits_workspace(int T, int d, int E);
moe_status router_logits(const uint16_t *x, const uint16_t *w, int T, int d, int E, float *logits, void *ws,
                         int32_t *dev_status, cudaStream_t st);
size_t router_backward_workspace(int T, int d, int E);
moe_status router_backward(const uint16_t *x, const uint16_t *w, const float *dl, int T, int d, int E, float *dx,
                           float *dw, void *ws, int32_t *dev_status, cudaStream_t st);

} // namespace moe
