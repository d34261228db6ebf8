#include "linear_internal.cuh"
namespace kda {
bool linear_tc_supported(int, int, DType) { return false; }
size_t linear_tc_scratch_bytes(int, int, int, int, long, int, bool, int) { return 0; }
cudaError_t launch_linear_tc(const LinFwd &, cudaStream_t) { return cudaErrorNotSupported; }
size_t linear_tc_bwd_scratch_bytes(int, int, int, int, int, int, int) { return 0; }
cudaError_t launch_linear_tc_bwd(const LinBwd &, cudaStream_t) { return cudaErrorNotSupported; }
}
