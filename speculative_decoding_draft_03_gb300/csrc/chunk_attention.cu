// chunk_attention.cu — attention of long blocks of queries (a chunk of a prompt) over a paged cache.
#include "serving.cuh"

namespace dspark {

size_t chunk_attention_scratch(int Hq, int Hkv, int D) { return attention_rows_scratch(Hq, Hkv, D); }

cudaError_t launch_chunk_attention(const AttentionArgs& a, void* scratch, cudaStream_t s) {
  return launch_attention_rows(a, scratch, s);
}

}  // namespace dspark
