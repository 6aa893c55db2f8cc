#include "csa_sparse_list.cuh"
namespace csa {
cudaError_t launch_sparse_backward(const SparseParams& p, int dtype, void* workspace, cudaStream_t stream) { return cudaErrorNotSupported; }
size_t sparse_backward_workspace(const SparseParams& p, int dtype) { return 256; }
cudaError_t take_status_sparse_bwd(uint32_t* out, cudaStream_t stream) { return take_status(out, stream); }
}
