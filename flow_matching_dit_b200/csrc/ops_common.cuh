// What the operator kernels share: the status word, 16-byte vectors of bf16
// and f32, and launches with programmatic dependent launch.
#pragma once

#include "host.cuh"
#include "ptx.cuh"

namespace gdit {

// Device status bits of the operators, beside DEV_ERR_TIMEOUT.
enum : unsigned {
  OP_ERR_GROUP = 8u,      // norm_residual: row_group out of range
  OP_ERR_OFFSETS = 16u,   // attention: bad sequence offsets or lengths
};

// One status word per device; kernels OR bits into it, gdit_op_status reads
// and clears them.
static __device__ unsigned g_op_status;

__device__ __forceinline__ float4 bf16x4_to_f32(uint2 v) {
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}

// Every operator kernel starts with pdl_wait() before it touches memory, and
// calls pdl_launch_dependents() only after that (and after its TMEM
// allocation), so at most two kernels of a stream are resident at a time and a
// waiting one never holds TMEM that the running one still has to get.
template <typename... KArgs, typename... Args>
void launch_op(cudaStream_t s, int cluster, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
               Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...));
}

}  // namespace gdit
