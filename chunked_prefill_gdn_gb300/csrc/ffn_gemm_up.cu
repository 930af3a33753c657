// ffn_gemm.cuh, the products that end in the up epilogue.
#include "ffn_gemm.cuh"

namespace gdn {
namespace ffn {
GDN_FFN_LAUNCHER(launch_up, kUp)
}  // namespace ffn
}  // namespace gdn
