// The fp32 kernels of kv4_decode.cuh.
#include "kv4_decode.cuh"

namespace rc {
namespace kv4 {

template cudaError_t launch<float>(const Params&, cudaStream_t);

}  // namespace kv4
}  // namespace rc
