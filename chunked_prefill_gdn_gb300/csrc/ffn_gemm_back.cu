// ffn_gemm.cuh, the products that end in the back epilogue.
#include "ffn_gemm.cuh"

namespace gdn {
namespace ffn {
GDN_FFN_LAUNCHER(launch_back, kBack)
}  // namespace ffn
}  // namespace gdn
