// Chunked linear attention, bf16 storage (kernel in linattn_kernel.h).
#include "linattn_inst.h"

namespace prism {
template hipError_t launch_la_pass<bf16>(const LaArgs<bf16>&, int, LaPass, hipStream_t);
}  // namespace prism
