// The planner of tile maps as a launch of its own (tile_plan.cuh).
#include "tile_plan.cuh"

namespace hpc {
namespace {

template <int T>
__global__ void __launch_bounds__(tileplan::kThreads) tile_plan_kernel(const TilePlanArgs a) {
    grid_dependency_wait();  // the lengths may come from the kernel before
    grid_launch_dependents();
    tileplan::tile_plan_block<T>(a);
}

}  // namespace

cudaError_t launch_tile_plan(const TilePlanArgs& a, cudaStream_t s) {
    return launch_pdl(a.T == kTilePair ? tile_plan_kernel<kTilePair> : tile_plan_kernel<kTileCta>, dim3(1),
                      dim3(tileplan::kThreads), 0, s, a);
}

}  // namespace hpc
