// query_page_128.cu -- the page-major query kernel at head_dim 128 (a file for each head_dim, so
// that they compile in parallel).
#include "query_page.cuh"

namespace kvq {

cudaError_t launch_query_pages_128(const QueryAttnParams& p, bool two, cudaStream_t s) {
  return two ? query_page_fmt<128, 2>(p, s) : query_page_fmt<128, 1>(p, s);
}

}  // namespace kvq
