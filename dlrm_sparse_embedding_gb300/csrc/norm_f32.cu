// Layer norm's kernels for f32 rows.
#define EMB_NORM_KERNELS
#include "norm.cuh"

namespace emb {
namespace norm {

template int launch_rows<float>(Args, int, bool, const Shape&, cudaStream_t);

}  // namespace norm
}  // namespace emb
