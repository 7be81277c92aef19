// query_page_256.cu -- the page-major query kernel at head_dim 256 (a file for each head_dim, so
// that they compile in parallel).
#include "query_page.cuh"

namespace kvq {

cudaError_t launch_query_pages_256(const QueryAttnParams& p, cudaStream_t s) { return query_page_fmt<256, 1>(p, s); }

}  // namespace kvq
