// Host-only stand-ins for the launchers that api_blocks.cpp calls, linked with
// it into a sanitizer build of its validation code (no device code).
#include "blocks.hpp"

namespace fp8bs {

int gated_few_cuts(int64_t M, int64_t N, int64_t K, bool) { return M > 64 ? 0 : N <= 2048 && K > 128 ? 2 : 1; }
int64_t gated_few_parts(int64_t M, int64_t N, int64_t K, bool, bool) { return 2 * gated_few_cuts(M, N, K, true); }
hipError_t launch_gated_few(const GatedFewProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_gated_backward(const GatedGradProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_head_norm_rotary(const HeadProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_head_norm_rotary_backward(const HeadProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
int64_t head_grad_parts(int64_t T, int64_t, int64_t, int64_t) { return T < 1024 ? T : 1024; }
hipError_t launch_quant_cols(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t,
                             float*, bool, hipStream_t) { return hipErrorInvalidDeviceFunction; }
hipError_t launch_gemm(const GemmProblem&, hipStream_t) { return hipErrorInvalidDeviceFunction; }
void attach_gemm_workspace(GemmProblem&, hipStream_t) {}

}  // namespace fp8bs
