// ffn_gemm.cuh, the products that end in the plain epilogue.
#include "ffn_gemm.cuh"

namespace gdn {
namespace ffn {
GDN_FFN_LAUNCHER(launch_plain, kPlain)
}  // namespace ffn
}  // namespace gdn
