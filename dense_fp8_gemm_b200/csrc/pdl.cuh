// Programmatic dependent launch for the library's element-wise kernels.
//
// A kernel launched with launch_pdl may start while the previous kernel in
// the stream is still running; it calls pdl_wait() before reading anything
// that kernel writes. It calls pdl_trigger() at entry, so the next kernel
// (a GEMM, which waits the same way before reading its activations) can take
// SMs as they free up and prefetch its weights meanwhile.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace spense {

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Loads of what an earlier grid writes. It may still run when this grid starts, so the
// data is not read-only as long as this kernel runs, which the non-coherent loads ask
// for (__ldg, and plain ones through const __restrict__ pointers). These are coherent, and
// volatile asm keeps its place behind pdl_wait(); so do plain loads through pointers
// without __restrict__, which pdl_wait()'s memory clobber holds back.
__device__ __forceinline__ uint32_t ld_dep(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int32_t ld_dep(const int32_t* p) {
  return static_cast<int32_t>(ld_dep(reinterpret_cast<const uint32_t*>(p)));
}
__device__ __forceinline__ long long ld_dep(const long long* p) {
  long long v;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint8_t ld_dep(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return static_cast<uint8_t>(v);
}
__device__ __forceinline__ uint2 ld_dep(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_dep(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ int4 ld_dep(const int4* p) {
  const uint4 v = ld_dep(reinterpret_cast<const uint4*>(p));
  return make_int4(static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w));
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), unsigned int grid, unsigned int block, size_t smem,
                       cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace spense
