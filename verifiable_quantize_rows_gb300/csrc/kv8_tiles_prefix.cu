// kv8_tiles_prefix.cu -- attention over a shared prefix of many query rows over the int8 cache.
#include <type_traits>

#include "kv8_more.h"
#include "kv8_tiles.cuh"

namespace bsg {

cudaError_t launch_tiles_prefix(const KvCall &a, const KvPlan &p, cudaStream_t st) { return launch_tiles<true>(a, p, st); }

}  // namespace bsg
