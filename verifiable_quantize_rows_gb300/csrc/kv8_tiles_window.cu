// kv8_tiles_window.cu -- attention through a window of many query rows over the int8 cache.
#include <type_traits>

#include "kv8_more.h"
#include "kv8_tiles.cuh"

namespace bsg {

cudaError_t launch_tiles_window(const KvCall &a, const KvPlan &p, cudaStream_t st) { return launch_tiles<false>(a, p, st); }

}  // namespace bsg
