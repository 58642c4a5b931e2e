// zmoe_add_rmsnorm: the residual addition, the RMSNorm of the sum and its 8-bit codes in one pass.
//
// ZONOS2 Technical Report digest, "method overview and architecture", item 5 (RMSNorm, pre-norm blocks),
// and the ZONOS2 page of the sglang-omni cookbook, "Benchmark Results" (the served model runs fp8).  Per row t:
//   h'[t] = h[t] + delta[t]                                     (fp32 sum, rounded to h's type)
//   x[t]  = h'[t] / sqrt(mean_c h'[t, c]^2 + eps) * gamma       (of the rounded h', in fp32)
//   s     = max|x| / 448 over a row, or over each 128 columns;  codes = E4M3 nearest x * fp32(1 / s)
// The codes take the unrounded fp32 x, so that they carry one rounding; x itself is rounded to its type
// once, on its way out.  The squares are summed in fp32 as they are: no row of a trained model comes near 2^64 or, without
// eps, 2^-56, and scaling such rows first cost 1 to 6% of every other row's time (a second sum behind a branch).
//
// Bound by HBM: h and delta are read once, h', x and the codes written once.  A row stays in its threads'
// registers between the two reductions (sum of squares, largest magnitude).  A thread takes chunks of CH
// neighbouring columns: 16 where h and delta are both bf16 (two 16-byte loads each; half the shuffles and scales a
// column that 8 take), 8 otherwise (an f32 chunk of 8 is two 16-byte loads already).  16-bit rows are bound by
// instructions and the L1 cache before they are by HBM, so a block takes several of them and keeps the gains in
// registers (5003 x 4096: 38.6 us with 8 columns, 30.7 with 16, 27.5 with the gains kept); f32 rows run at the copy
// rate with a block a row, and lost by the registers that a loop takes (72 to 75 us).
//
// Measured: 16384 x 2048, f32 in, f32, bf16 and codes out: 80 us, 6.2 TB/s; 5003 x 4096, bf16 in and out, codes in
// blocks of 128: 27.5 us, 5.2 TB/s; one row of 2048: 4.2 us a call, which is the host's time.
#include "vectors.cuh"

namespace zmoe {
namespace {

constexpr char kName[] = "zmoe_add_rmsnorm";
constexpr int kRowThreads = 512;   // threads a row is spread over at most
constexpr int kMaxD = 32768;       // 512 threads with 64 columns each

struct AddNormArgs {
  const void* h;
  const void* delta;    // or null
  const float* gamma;
  float eps, inv_d;
  int T, d;
  int group;            // columns per scale: 0 = the row, 128
  void* h_out;          // or null
  void* x;              // or null
  uint8_t* codes;       // or null
  float* scales;
};

// The scale of values whose largest magnitude is amax; never so small that its reciprocal overflows.
__device__ __forceinline__ float code_scale(float amax) {
  return amax > 0.f ? fmaxf(__fdiv_rn(amax, 448.f), 1.17549435e-38f) : 1.f;
}

// One row per blockDim.x threads (a multiple of 32), blockDim.y rows per block at a time.
template <typename TH, typename TD, typename TX, int CH, int N>
__global__ void __launch_bounds__(kRowThreads) add_rmsnorm_kernel(AddNormArgs a) {
  constexpr int kVecs = CH / 8;      // vectors of 8 columns a chunk
  constexpr bool kKeep = CH == 16 && N == 1;   // the gains stay in registers from row to row
  __shared__ float red[2][2][kRowThreads / 32];   // [row parity][sum, largest]
  enter_behind();
  const int warps_row = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = threadIdx.x * CH, step = blockDim.x * CH;
  float kept[kKeep ? kVecs : 1][8];
  auto gains = [&](int c, float* g) {
    const float4 g0 = *reinterpret_cast<const float4*>(a.gamma + c);
    const float4 g1 = reinterpret_cast<const float4*>(a.gamma + c)[1];
    g[0] = g0.x; g[1] = g0.y; g[2] = g0.z; g[3] = g0.w;
    g[4] = g1.x; g[5] = g1.y; g[6] = g1.z; g[7] = g1.w;
  };
  if (kKeep) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      if (c0 + 8 * k < a.d) gains(c0 + 8 * k, kept[k]);
  }
  int parity = 0;
  for (long long first = static_cast<long long>(blockIdx.x) * blockDim.y; first < a.T;
       first += static_cast<long long>(gridDim.x) * blockDim.y, parity ^= 1) {
    float* sums = red[parity][0] + threadIdx.y * warps_row;
    float* tops = red[parity][1] + threadIdx.y * warps_row;
    const long long row = first + threadIdx.y;
    const size_t base = static_cast<size_t>(row < a.T ? row : 0) * a.d;
    const int end = row < a.T ? a.d : 0;   // columns from here on are not there
    const TH* h = static_cast<const TH*>(a.h) + base;
    const TD* dl = static_cast<const TD*>(a.delta) + base;
    Raw8<TH> raw[N][kVecs];
    float v[N][kVecs][8];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = c0 + i * step + 8 * k;
        if (c < end) raw[i][k].load(h + c);
        else raw[i][k].clear();
      }
    if (a.delta) {
      Raw8<TD> add[N][kVecs];
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int c = c0 + i * step + 8 * k;
          if (c < end) add[i][k].load(dl + c);
          else add[i][k].clear();
        }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          float w[8];
          raw[i][k].get(v[i][k]);
          add[i][k].get(w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][k][e] += w[e];
          raw[i][k].put(v[i][k]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) raw[i][k].get(v[i][k]);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = c0 + i * step + 8 * k;
        if (a.h_out && c < end) raw[i][k].store(static_cast<TH*>(a.h_out) + base + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][k][e], v[i][k][e], ss);
      }
    ss = warp_sum(ss);
    if (warps_row > 1) {
      if (lane == 0) sums[warp] = ss;
      __syncthreads();
      ss = warp_sum(lane < warps_row ? sums[lane] : 0.f);
    }
    const float inv = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    float amax[N];   // of a chunk
#pragma unroll
    for (int i = 0; i < N; ++i) {
      amax[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const int c = c0 + i * step + 8 * k;
        if (c < end) {
          float g[8];
          if (!kKeep) gains(c, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[i][k][e] = v[i][k][e] * inv * (kKeep ? kept[kKeep ? k : 0][e] : g[e]);
            amax[i] = fmaxf(amax[i], fabsf(v[i][k][e]));
          }
          if (a.x) store8(static_cast<TX*>(a.x) + base + c, v[i][k]);
        }
      }
    }
    if (!a.codes) {   // uniform over the grid
      if (!kKeep) return;
      continue;
    }
    if (a.group == 0) {
      float top = amax[0];
#pragma unroll
      for (int i = 1; i < N; ++i) top = fmaxf(top, amax[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (warps_row > 1) {
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        top = lane < warps_row ? tops[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const float s = code_scale(top), r = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
          const int c = c0 + i * step + 8 * k;
          if (c < end)
            *reinterpret_cast<uint2*>(a.codes + base + c) = make_uint2(e4m3x4(v[i][k], r), e4m3x4(v[i][k] + 4, r));
        }
      if (row < a.T && threadIdx.x == 0) a.scales[row] = s;
    } else {   // 128 columns = 128 / CH neighbouring lanes
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = c0 + i * step;
        float top = amax[i];
#pragma unroll
        for (int o = 64 / CH; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (c < end) {   // d % 128 == 0: whole chunks
          const float s = code_scale(top), r = __frcp_rn(s);
          uint32_t w[2 * kVecs];
#pragma unroll
          for (int k = 0; k < 2 * kVecs; ++k) w[k] = e4m3x4(v[i][k >> 1] + 4 * (k & 1), r);
          if (kVecs == 2)
            *reinterpret_cast<uint4*>(a.codes + base + c) = make_uint4(w[0], w[1], w[2 * kVecs - 2], w[2 * kVecs - 1]);
          else
            *reinterpret_cast<uint2*>(a.codes + base + c) = make_uint2(w[0], w[1]);
          if ((c & 127) == 0) a.scales[static_cast<size_t>(row) * (a.d >> 7) + (c >> 7)] = s;
        }
      }
    }
    if (!kKeep) return;   // one row a block
  }
}

// Chunks a thread holds: one as long as 256 threads reach a row's end.
template <typename TH, typename TD, typename TX, int CH>
zmoe_status launch_row(const AddNormArgs& a, cudaStream_t s) {
  const int chunks = (a.d + CH - 1) / CH;
  int n = 1;
  while (chunks > 256 * n && n * CH < 64) n *= 2;
  const int threads = ((chunks + n - 1) / n + 31) / 32 * 32;
  const dim3 block(threads, threads >= 256 ? 1 : 256 / threads);
  int grid = (a.T + block.y - 1) / block.y;
  if (CH == 16 && n == 1) {   // several rows a block (kKeep), as many for each
    const int most = num_sms() * 4;
    grid = (grid + (grid + most - 1) / most - 1) / ((grid + most - 1) / most);
  }
  switch (n) {
    case 1: return launch_behind(kName, add_rmsnorm_kernel<TH, TD, TX, CH, 1>, dim3(grid), block, 0, s, 1, a);
    case 2: return launch_behind(kName, add_rmsnorm_kernel<TH, TD, TX, CH, 2>, dim3(grid), block, 0, s, 1, a);
    case 4: return launch_behind(kName, add_rmsnorm_kernel<TH, TD, TX, CH, 4>, dim3(grid), block, 0, s, 1, a);
    default: return launch_behind(kName, add_rmsnorm_kernel<TH, TD, TX, CH, 64 / CH>, dim3(grid), block, 0, s, 1, a);
  }
}

template <typename TH, typename TD>
zmoe_status launch_x(const AddNormArgs& a, zmoe_dtype xt, cudaStream_t s) {
  constexpr int CH = sizeof(TH) + sizeof(TD) == 4 ? 16 : 8;
  return xt == ZMOE_BF16 ? launch_row<TH, TD, uint16_t, CH>(a, s) : launch_row<TH, TD, float, CH>(a, s);
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
  ZMOE_REQUIRE(!delta || h_out != delta || h_dtype == delta_dtype,
               "zmoe_add_rmsnorm: h_out may be delta only where their types are one");
  if (d > kMaxD) return fail(ZMOE_ERR_UNSUPPORTED, "zmoe_add_rmsnorm: d must be at most 32768");
  clear_error();
  const AddNormArgs a{h, delta, gamma, eps, 1.f / static_cast<float>(d), T, d, group, h_out, x, codes, scales};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (h_dtype == ZMOE_BF16)
    return delta_dtype == ZMOE_BF16 ? launch_x<uint16_t, uint16_t>(a, x_dtype, s) : launch_x<uint16_t, float>(a, x_dtype, s);
  return delta_dtype == ZMOE_BF16 ? launch_x<float, uint16_t>(a, x_dtype, s) : launch_x<float, float>(a, x_dtype, s);
}
