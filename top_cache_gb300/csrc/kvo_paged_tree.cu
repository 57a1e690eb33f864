// The kernel of the attention over 16 and 4 bits (kvo_paged_attend.cuh) where the
// query tokens are the nodes of a tree.
#include "kvo_paged_attend.cuh"

namespace kvo {

cudaError_t launch_paged_tree(const PagedAttendArgs& a, int N, bool q4, cudaStream_t s) {
  return launch_attend<true>(a, N, q4, s);
}

}  // namespace kvo
