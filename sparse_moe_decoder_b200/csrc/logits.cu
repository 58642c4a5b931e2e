// zmoe_adjust_logits: penalties for repeated ids, biases and a mask of allowed ids on the codebook logits, and
// the greedy id of the adjusted row.
//
// ZONOS2 page of the sglang-omni cookbook, request parameters (repetition penalty); ZONOS2 Technical Report
// digest, "method overview and architecture", items 1 and 5 (the next frame of the delay-patterned codebooks).
// With c the occurrences of id v of codebook n in the stream's history, each step rounded to fp32:
//   l <- c > 0 ? (l > 0 ? l / r : l * r) : l;   l <- l - f c;   l <- c > 0 ? l - p : l;   l <- l + bias
//   l <- -inf where the mask forbids v;   out = l rounded to its type;   id = the largest out's lowest id
//
// Bound by HBM for large vocabularies (logits read once, written once), by latency for one frame.  A row
// (stream, codebook) is split over a cluster of 1 to 8 CTAs.  Each counts its ids' occurrences in shared memory
// (16-bit counters, so up to 32768 ids a pass), passes over its logits once, and leaves its best (value, id) in
// the first CTA's shared memory, which takes the largest: no workspace, one launch, and the order in which CTAs
// finish does not matter.
#include "sm100_ptx.cuh"

namespace zmoe {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSplit = 8;       // the portable cluster size
constexpr int kChunk = 32768;      // ids counted at a time
constexpr int kMaxHistory = 65535; // what a 16-bit counter holds

struct AdjustArgs {
  const void* logits;
  void* out;
  const int32_t* history;     // [T, L, N] or null
  const int32_t* hist_lens;   // [T] or null
  const float *repetition, *presence, *frequency;   // [T] or null
  const float* bias;          // [N, V] or null
  const uint32_t* mask;       // [T, N, ceil(V / 32)] or null
  int32_t* ids;               // [T, N] or null
  int N, V, L, split, range;  // range: ids per CTA, a multiple of 32
  unsigned int* errors;
};

// Plain loads: `out` may be `logits`.
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
// The stored value, as fp32.
__device__ __forceinline__ float store1(float* p, float v) { *p = v; return v; }
__device__ __forceinline__ float store1(uint16_t* p, float v) {
  const uint16_t b = f32_to_bf16_bits(v);
  *p = b;
  return bf16_to_f32(b);
}

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// (value, id) pairs: the larger value wins, then the lower id.  -1 (as unsigned, the highest) is no id.
__device__ __forceinline__ void take(float& v, uint32_t& i, float w, uint32_t j) {
  if (j != 0xFFFFFFFFu && (i == 0xFFFFFFFFu || w > v || (w == v && j < i))) {
    v = w;
    i = j;
  }
}

template <typename TL>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustArgs a) {
  extern __shared__ uint32_t counts[];   // 16-bit counters, two a word
  __shared__ float best_v[kWarps];
  __shared__ uint32_t best_i[kWarps];
  __shared__ unsigned long long part[kMaxSplit];
  const int rank = blockIdx.x % a.split, row = blockIdx.x / a.split;   // row = t * N + n
  const int t = row / a.N, n = row - t * a.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long base = static_cast<long long>(row) * a.V;
  const TL* src = static_cast<const TL*>(a.logits) + base;
  TL* dst = static_cast<TL*>(a.out) + base;
  const float* bias = a.bias ? a.bias + static_cast<size_t>(n) * a.V : nullptr;
  const uint32_t* mask = a.mask ? a.mask + static_cast<size_t>(row) * ((a.V + 31) / 32) : nullptr;
  const bool counted = a.history != nullptr;
  int len = 0;
  if (counted) {
    len = a.hist_lens ? a.hist_lens[t] : a.L;
    len = len < 0 ? 0 : (len > a.L ? a.L : len);
  }
  const float rep = a.repetition ? a.repetition[t] : 1.f, pre = a.presence ? a.presence[t] : 0.f,
              frq = a.frequency ? a.frequency[t] : 0.f;
  const int32_t* hist = counted ? a.history + static_cast<size_t>(t) * a.L * a.N + n : nullptr;
  const int v_begin = rank * a.range;
  const int v_end = v_begin + a.range < a.V ? v_begin + a.range : a.V;
  float bv = 0.f;
  uint32_t bi = 0xFFFFFFFFu;
  for (int c0 = v_begin; c0 < v_end; c0 += kChunk) {
    const int c1 = v_end - c0 < kChunk ? v_end : c0 + kChunk;
    if (counted) {
      __syncthreads();   // the previous chunk's counts are read
      for (int i = threadIdx.x; i < (c1 - c0 + 1) / 2; i += kThreads) counts[i] = 0u;
      __syncthreads();
#pragma unroll 4
      for (int i = threadIdx.x; i < len; i += kThreads) {
        const int id = __ldg(hist + static_cast<size_t>(i) * a.N);
        if (id >= c0 && id < c1) atomicAdd(&counts[(id - c0) >> 1], 1u << (((id - c0) & 1) * 16));
        if (id >= a.V && rank == 0 && c0 == 0) record_device_error(a.errors);   // a negative id is no id
      }
      __syncthreads();
    }
#pragma unroll 4
    for (int v = c0 + static_cast<int>(threadIdx.x); v < c1; v += kThreads) {
      float l = load1(src + v);
      if (counted) {
        const uint32_t c = (counts[(v - c0) >> 1] >> (((v - c0) & 1) * 16)) & 0xFFFFu;
        if (c) {
          if (a.repetition) l = l > 0.f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
          if (a.frequency) l = __fsub_rn(l, __fmul_rn(frq, static_cast<float>(c)));
          if (a.presence) l = __fsub_rn(l, pre);
        }
      }
      if (bias) l = __fadd_rn(l, __ldg(bias + v));
      const bool ok = !mask || ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u);
      if (!ok) l = __int_as_float(0xff800000);
      const float w = store1(dst + v, l);
      if (ok && w == w) take(bv, bi, w, static_cast<uint32_t>(v));   // NaN never wins
    }
  }
  if (!a.ids) return;   // uniform over the grid
  // the first CTA of the cluster runs before any other writes to it
  if (a.split > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, bv, o);
    const uint32_t j = __shfl_xor_sync(0xffffffffu, bi, o);
    take(bv, bi, w, j);
  }
  if (lane == 0) {
    best_v[warp] = bv;
    best_i[warp] = bi;
  }
  __syncthreads();
  if (a.split > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) take(bv, bi, best_v[w], best_i[w]);
    if (a.split == 1) {
      a.ids[row] = static_cast<int32_t>(bi);   // -1: nothing allowed
    } else {
      const unsigned long long p = (static_cast<unsigned long long>(__float_as_uint(bv)) << 32) | bi;
      st_cluster_u64(mapa_shared(smem_u32(&part[rank]), 0), p);
    }
  }
  if (a.split > 1) {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (rank == 0 && threadIdx.x == 0) {
      float v = 0.f;
      uint32_t i = 0xFFFFFFFFu;
      for (int r = 0; r < a.split; ++r)
        take(v, i, __uint_as_float(static_cast<uint32_t>(part[r] >> 32)), static_cast<uint32_t>(part[r]));
      a.ids[row] = static_cast<int32_t>(i);
    }
  }
}

template <typename TL>
zmoe_status launch(const AdjustArgs& a, int rows, size_t smem, cudaStream_t s) {
  if (smem > 40 * 1024 && cudaFuncSetAttribute(adjust_kernel<TL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kChunk * 2 + 16) != cudaSuccess)
    return check_launch("zmoe_adjust_logits: shared memory attribute");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * a.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, adjust_kernel<TL>, a);
  return check_launch("zmoe_adjust_logits");
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace zmoe

extern "C" zmoe_status zmoe_adjust_logits(const void* logits, zmoe_dtype dtype, const int32_t* history,
                                          const int32_t* hist_lens, const float* repetition, const float* presence,
                                          const float* frequency, const float* bias, const uint32_t* mask, int T, int N,
                                          int V, int L, void* out, int32_t* ids, zmoe_stream_t stream) {
  ZMOE_TRACE("zmoe_adjust_logits");
  using namespace zmoe;
  ZMOE_REQUIRE(dtype_ok(dtype), "zmoe_adjust_logits: bad dtype");
  ZMOE_REQUIRE(T >= 0 && N >= 1 && V >= 1 && L >= 0, "zmoe_adjust_logits: T >= 0, N >= 1, V >= 1, L >= 0");
  ZMOE_REQUIRE(L <= kMaxHistory, "zmoe_adjust_logits: at most 65535 frames of history");
  ZMOE_REQUIRE(V <= 0x7fff0000, "zmoe_adjust_logits: V too large");
  if (T == 0) return ZMOE_OK;
  ZMOE_REQUIRE(logits && out, "zmoe_adjust_logits: NULL pointer");
  ZMOE_REQUIRE(history || !(repetition || presence || frequency || hist_lens),
               "zmoe_adjust_logits: penalties need a history");
  ZMOE_REQUIRE((reinterpret_cast<uintptr_t>(logits) & (dtype_size(dtype) - 1)) == 0 &&
                   (reinterpret_cast<uintptr_t>(out) & (dtype_size(dtype) - 1)) == 0 && aligned4(history) &&
                   aligned4(hist_lens) && aligned4(repetition) && aligned4(presence) && aligned4(frequency) &&
                   aligned4(bias) && aligned4(mask) && aligned4(ids),
               "zmoe_adjust_logits: misaligned pointer");
  const long long rows = static_cast<long long>(T) * N;
  ZMOE_REQUIRE(rows * kMaxSplit <= 0x7fffffffLL, "zmoe_adjust_logits: T * N too large");
  clear_error();
  AdjustArgs a{};
  a.logits = logits; a.out = out;
  a.history = (repetition || presence || frequency) && L > 0 ? history : nullptr;
  a.hist_lens = hist_lens;
  a.repetition = repetition; a.presence = presence; a.frequency = frequency;
  a.bias = bias; a.mask = mask; a.ids = ids;
  a.N = N; a.V = V; a.L = L;
  a.errors = device_error_counter();
  // enough CTAs for the machine, but at least 2048 ids each
  int split = 1;
  while (split < kMaxSplit && rows * split < 3LL * num_sms() && V / (2 * split) >= 2048) split *= 2;
  a.split = split;
  a.range = ((V + split - 1) / split + 31) / 32 * 32;
  const int ids_at_once = a.range < kChunk ? a.range : kChunk;
  const size_t smem = a.history ? static_cast<size_t>(ids_at_once) * 2 + 16 : 16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == ZMOE_BF16 ? launch<uint16_t>(a, static_cast<int>(rows), smem, s)
                            : launch<float>(a, static_cast<int>(rows), smem, s);
}
