// Layer norm's kernels for bf16 rows.
#define EMB_NORM_KERNELS
#include "norm.cuh"

namespace emb {
namespace norm {

template int launch_rows<__nv_bfloat16>(Args, int, bool, const Shape&, cudaStream_t);

}  // namespace norm
}  // namespace emb
