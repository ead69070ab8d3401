// Host-only stand-ins for the launchers that api_layers.cpp calls, linked with
// it into a sanitizer build of its validation code (no device code).
#include "layers.hpp"

namespace fp8bs {

hipError_t launch_layer_norm(const LayerNormProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_layer_norm_backward(const LayerNormGradProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
int64_t layer_norm_grad_parts(int64_t rows, int64_t) { return rows < 512 ? rows : 512; }
hipError_t launch_moe_few_tokens(const MoeProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_adapter_few(const AdapterProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_adapter_prompt(const AdapterProblem&, int64_t, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_gemm(const GemmProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
void attach_gemm_workspace(GemmProblem&, hipStream_t) {}

}  // namespace fp8bs
