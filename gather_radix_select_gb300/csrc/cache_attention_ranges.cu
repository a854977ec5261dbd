// cache_attention_ranges.cu -- the attention kernels whose positions are ranges: a window and the first tokens, a prefix
// shared by all sequences and what follows it.  (A file of its own: compiled beside the others.)
#include "cache_attention.cuh"

namespace sel {

cudaError_t launch_attention_ranges(const Kargs &k, cudaStream_t s) { return launch_layout<true>(k, s); }

}  // namespace sel
