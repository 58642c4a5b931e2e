// What the decode-step operators share: how they are launched, and vectors of values in memory and in fp32.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace zmoe {

// A decode step is a chain of kernels of a few microseconds.  Each is launched while the one before it still runs
// (programmatic dependent launch) and waits at its first line until that one is complete and its writes are visible,
// so that the launch itself is hidden: 1 to 2 us a kernel (the logits of one frame 6.1 to 4.3 us, attention of one
// stream 10.2 to 8.3).  Such a kernel touches no memory before the wait, and reads its inputs by plain loads: what the
// kernel before wrote is no read-only data of a kernel that began beside it.
template <typename... P, typename... A>
inline zmoe_status launch_behind(const char* what, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t stream, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kernel, args...);
  return check_launch(what);
}

// The first line of a kernel launched behind another: the next may be launched, and the one before is complete.
__device__ __forceinline__ void enter_behind() {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

// Two fp32 values rounded to bf16 by one instruction.
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void widen_bf16x2(uint32_t w, float* v) {
  v[0] = __uint_as_float(w << 16);
  v[1] = __uint_as_float(w & 0xFFFF0000u);
}

// E4M3 codes of four values times r (each product rounded to fp32; nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t e4m3x4(const float* v, float r) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[0], r), __fmul_rn(v[1], r)), __NV_SATFINITE,
                                              __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[2], r), __fmul_rn(v[3], r)), __NV_SATFINITE,
                                              __NV_E4M3);
  return __byte_perm(a, b, 0x5410);
}

// Eight neighbouring values as they lie in memory (16-byte aligned), and as fp32.
template <typename T>
struct Raw8;

template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  // The rounding to the type, kept in v too.
  __device__ __forceinline__ void put(float* v) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

template <>
struct Raw8<uint16_t> {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float* v) const {
    widen_bf16x2(a.x, v);
    widen_bf16x2(a.y, v + 2);
    widen_bf16x2(a.z, v + 4);
    widen_bf16x2(a.w, v + 6);
  }
  __device__ __forceinline__ void put(float* v) {
    a = make_uint4(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]), round_bf16x2(v[4], v[5]),
                   round_bf16x2(v[6], v[7]));
    get(v);
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  Raw8<T> r;
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = v[e];
  r.put(w);
  r.store(p);
}

}  // namespace zmoe
