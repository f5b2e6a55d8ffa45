// The paged attention's launch for few short items: a cluster of blocks for each.
#include <cuda_runtime.h>

#include "paged_attn_kernel.cuh"

namespace ditattn {
namespace paged {

cudaError_t launch_few(const PagedParams& p, int d, int rows, bool f32, int items, cudaStream_t st) {
  return for_sizes(d, rows, f32, [&](auto D, auto nb, auto zero) {
    using OT = decltype(zero);
    const cudaError_t e = prepare_kernel<D(), nb(), OT, true>();
    if (e != cudaSuccess) return e;
    return launch_after<kCluster>(paged_attn_kernel<D(), nb(), OT, true>, dim3(items * kCluster), dim3(kThreadsPaged),
                                  PagedSmem<D()>::bytes(nb()), st, p);
  });
}

}  // namespace paged
}  // namespace ditattn
