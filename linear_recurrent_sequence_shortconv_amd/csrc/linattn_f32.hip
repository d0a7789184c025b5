// Chunked linear attention, f32 storage (kernel in linattn_kernel.h).
#include "linattn_inst.h"

namespace prism {
template hipError_t launch_la_pass<float>(const LaArgs<float>&, int, LaPass, hipStream_t);
}  // namespace prism
