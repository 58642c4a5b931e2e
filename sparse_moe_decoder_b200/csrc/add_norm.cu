// zmoe_add_rmsnorm: the residual addition, the RMSNorm of the sum and its 8-bit codes in one pass.
//
// ZONOS2 Technical Report digest, "method overview and architecture", item 5 (RMSNorm, pre-norm blocks),
// and the ZONOS2 page of the sglang-omni cookbook, "Benchmark Results" (the served model runs fp8).  Per row t:
//   h'[t] = h[t] + delta[t]                                     (fp32 sum, rounded to h's type)
//   x[t]  = h'[t] / sqrt(mean_c h'[t, c]^2 + eps) * gamma       (of the rounded h', in fp32)
//   s     = max|x| / 448 over a row, or over each 128 columns;  codes = E4M3 nearest x * fp32(1 / s)
// The codes take the unrounded fp32 x, so that they carry one rounding; x itself is rounded to its type
// once, on its way out.
//
// Bound by HBM: h and delta are read once, h', x and the codes written once.  A row stays in its threads'
// registers between the two reductions (sum of squares, largest magnitude), 8 columns (one 16-byte load of
// bf16, two of f32) a vector, VPT vectors a thread.
#include <cuda_fp8.h>

#include "common.cuh"

namespace zmoe {
namespace {

constexpr int kMaxVpt = 8;
constexpr int kRowThreads = 512;   // threads a row is spread over at most
constexpr int kMaxD = kRowThreads * kMaxVpt * 8;

struct AddNormArgs {
  const void* h;
  const void* delta;    // or null
  const float* gamma;
  float eps;
  int T, d;
  int tpr;              // threads per row (a multiple of 32)
  int group;            // columns per scale: 0 = the row, 128
  void* h_out;          // or null
  void* x;              // or null
  uint8_t* codes;       // or null
  float* scales;
};

__device__ __forceinline__ void load8(const uint16_t* p, float* v) { unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v); }

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float round_to(uint16_t*, float v) { return bf16_to_f32(f32_to_bf16_bits(v)); }
__device__ __forceinline__ float round_to(float*, float v) { return v; }

// The scale of values whose largest magnitude is amax; never so small that its reciprocal overflows.
__device__ __forceinline__ float code_scale(float amax) {
  return amax > 0.f ? fmaxf(__fdiv_rn(amax, 448.f), 1.17549435e-38f) : 1.f;
}

__device__ __forceinline__ uint2 encode8(const float* v, float r) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i], r), __fmul_rn(v[4 * i + 1], r)),
                                                __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i + 2], r), __fmul_rn(v[4 * i + 3], r)),
                                                __NV_SATFINITE, __NV_E4M3);
    w[i] = (a & 0xFFFFu) | (b << 16);
  }
  return make_uint2(w[0], w[1]);
}

// One row per tpr threads; blockDim.x / tpr rows per block.
template <typename TH, typename TD, typename TX, int VPT>
__global__ void __launch_bounds__(kRowThreads) add_rmsnorm_kernel(AddNormArgs a) {
  __shared__ float red[2][kRowThreads / 32];
  const int warps_row = a.tpr >> 5;
  const int r_in_block = threadIdx.x / a.tpr, t_in_row = threadIdx.x - r_in_block * a.tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * (blockDim.x / a.tpr) + r_in_block;
  const int vecs = a.d >> 3;
  const bool live = row < a.T;
  const size_t base = static_cast<size_t>(live ? row : 0) * a.d;
  const TH* h = static_cast<const TH*>(a.h) + base;
  const TD* dl = static_cast<const TD*>(a.delta) + base;
  float v[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t_in_row + i * a.tpr) * 8;
    const bool on = live && c < a.d;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    if (on) load8(h + c, v[i]);
  }
  if (a.delta) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t_in_row + i * a.tpr) * 8;
      if (live && c < a.d) {
        float w[8];
        load8(dl + c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = round_to(static_cast<TH*>(nullptr), v[i][e] + w[e]);
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t_in_row + i * a.tpr) * 8;
    if (a.h_out && live && c < a.d) store8(static_cast<TH*>(a.h_out) + base + c, v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
  }
  ss = warp_sum(ss);
  if (warps_row > 1) {
    if (lane == 0) red[0][warp] = ss;
    __syncthreads();
    ss = warp_sum(lane < warps_row ? red[0][r_in_block * warps_row + lane] : 0.f);
  }
  const float inv = rsqrtf(ss / static_cast<float>(a.d) + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t_in_row + i * a.tpr) * 8;
    if (live && c < a.d) {
      float g[8];
      load8(a.gamma + c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = v[i][e] * inv * g[e];
        amax = fmaxf(amax, fabsf(v[i][e]));
      }
      if (a.x) store8(static_cast<TX*>(a.x) + base + c, v[i]);
    }
  }
  if (!a.codes) return;   // uniform over the grid
  if (a.group == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (warps_row > 1) {
      if (lane == 0) red[1][warp] = amax;
      __syncthreads();
      amax = lane < warps_row ? red[1][r_in_block * warps_row + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    const float s = code_scale(amax), r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t_in_row + i * a.tpr) * 8;
      if (live && c < a.d) *reinterpret_cast<uint2*>(a.codes + base + c) = encode8(v[i], r);
    }
    if (live && t_in_row == 0) a.scales[row] = s;
  } else {   // 128 columns = 16 neighbouring lanes
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int vec = t_in_row + i * a.tpr, c = vec * 8;
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[i][e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (live && vec < vecs) {
        const float s = code_scale(m);
        *reinterpret_cast<uint2*>(a.codes + base + c) = encode8(v[i], __frcp_rn(s));
        if ((vec & 15) == 0) a.scales[static_cast<size_t>(row) * (a.d >> 7) + (vec >> 4)] = s;
      }
    }
  }
}

template <typename TH, typename TD, typename TX>
void launch_vpt(const AddNormArgs& a, int vpt, int block, int grid, cudaStream_t s) {
  switch (vpt) {
    case 1: add_rmsnorm_kernel<TH, TD, TX, 1><<<grid, block, 0, s>>>(a); break;
    case 2: add_rmsnorm_kernel<TH, TD, TX, 2><<<grid, block, 0, s>>>(a); break;
    case 4: add_rmsnorm_kernel<TH, TD, TX, 4><<<grid, block, 0, s>>>(a); break;
    default: add_rmsnorm_kernel<TH, TD, TX, 8><<<grid, block, 0, s>>>(a); break;
  }
}

template <typename TH, typename TD>
void launch_x(const AddNormArgs& a, zmoe_dtype xt, int vpt, int block, int grid, cudaStream_t s) {
  if (xt == ZMOE_BF16) launch_vpt<TH, TD, uint16_t>(a, vpt, block, grid, s);
  else launch_vpt<TH, TD, float>(a, vpt, block, grid, s);
}

}  // namespace
}  // namespace zmoe

extern "C" zmoe_status zmoe_add_rmsnorm(const void* h, zmoe_dtype h_dtype, const void* delta, zmoe_dtype delta_dtype,
                                        const float* gamma, float eps, int T, int d, void* h_out, void* x,
                                        zmoe_dtype x_dtype, uint8_t* codes, float* scales, int group,
                                        zmoe_stream_t stream) {
  ZMOE_TRACE("zmoe_add_rmsnorm");
  using namespace zmoe;
  ZMOE_REQUIRE(dtype_ok(h_dtype) && dtype_ok(delta_dtype) && dtype_ok(x_dtype), "zmoe_add_rmsnorm: bad dtype");
  ZMOE_REQUIRE(T >= 0, "zmoe_add_rmsnorm: T must be >= 0");
  ZMOE_REQUIRE(d >= 8 && d % 8 == 0, "zmoe_add_rmsnorm: d must be a positive multiple of 8");
  ZMOE_REQUIRE(eps >= 0.f, "zmoe_add_rmsnorm: eps must be >= 0");
  ZMOE_REQUIRE(group == 0 || group == 128, "zmoe_add_rmsnorm: group must be 0 (a scale per row) or 128");
  ZMOE_REQUIRE(group == 0 || d % 128 == 0, "zmoe_add_rmsnorm: group 128 needs d % 128 == 0");
  if (T == 0) return ZMOE_OK;
  ZMOE_REQUIRE(h && gamma, "zmoe_add_rmsnorm: NULL pointer");
  ZMOE_REQUIRE(h_out || x || codes, "zmoe_add_rmsnorm: no output asked for");
  ZMOE_REQUIRE((codes != nullptr) == (scales != nullptr), "zmoe_add_rmsnorm: codes and scales come together");
  ZMOE_REQUIRE(aligned16(h) && aligned16(gamma) && (!delta || aligned16(delta)) && (!h_out || aligned16(h_out)) &&
                   (!x || aligned16(x)) && (!codes || aligned16(codes)) &&
                   (reinterpret_cast<uintptr_t>(scales) & 3u) == 0,
               "zmoe_add_rmsnorm: pointers must be 16-byte aligned (scales: 4-byte)");
  if (d > kMaxD) return fail(ZMOE_ERR_UNSUPPORTED, "zmoe_add_rmsnorm: d must be at most 32768");
  clear_error();
  const int vecs = d / 8;
  int vpt = 1;
  while (vecs > kRowThreads * vpt) vpt *= 2;
  int tpr = (vecs + vpt - 1) / vpt;
  tpr = (tpr + 31) / 32 * 32;
  const int rows = tpr >= 256 ? 1 : 256 / tpr;
  AddNormArgs a{h, delta, gamma, eps, T, d, tpr, group, h_out, x, codes, scales};
  const int grid = (T + rows - 1) / rows, block = rows * tpr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (h_dtype == ZMOE_BF16) {
    if (delta_dtype == ZMOE_BF16) launch_x<uint16_t, uint16_t>(a, x_dtype, vpt, block, grid, s);
    else launch_x<uint16_t, float>(a, x_dtype, vpt, block, grid, s);
  } else {
    if (delta_dtype == ZMOE_BF16) launch_x<float, uint16_t>(a, x_dtype, vpt, block, grid, s);
    else launch_x<float, float>(a, x_dtype, vpt, block, grid, s);
  }
  return check_launch("zmoe_add_rmsnorm");
}
