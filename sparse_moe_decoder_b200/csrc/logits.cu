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
//
// The pass takes four neighbouring logits at an aligned address a thread at a time, two such vectors in flight; the
// first ones are on their way before the counting starts.  Rows of odd length start anywhere in a vector, so a
// vector's ids begin at 4 i - shift and the counters are laid out by id + shift; the vectors at a row's two ends go
// element by element, so nothing outside the row is touched.
//
// The pass leaves out the ids that were counted.  Few as they are, most warps hold one of them, and would take
// every step of the penalties for it; instead each is listed when its count leaves zero, and a thread of its own
// takes it.
#include "sm100_ptx.cuh"
#include "vectors.cuh"

namespace zmoe {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 2;          // vectors of four logits in flight a thread
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
  int N, V, L, split;
  int at_once;                // vectors counted at a time
  int same;                   // logits and out lie alike within a vector
  unsigned int* errors;
};

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return bf16_to_f32(v); }
// Plain loads: `out` may be `logits`.
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xFFFF0000u);
  v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xFFFF0000u);
}
// Four values rounded to the type (and v to what is stored).
template <typename TL>
struct Out4;
template <>
struct Out4<float> {
  float4 w;
  __device__ __forceinline__ void round(float* v) { w = make_float4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
  __device__ __forceinline__ void store_one(float* p, int e) const { *p = e == 0 ? w.x : (e == 1 ? w.y : (e == 2 ? w.z : w.w)); }
};
template <>
struct Out4<uint16_t> {
  uint2 w;
  __device__ __forceinline__ void round(float* v) {
    w = make_uint2(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
    widen_bf16x2(w.x, v);
    widen_bf16x2(w.y, v + 2);
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = w; }
  __device__ __forceinline__ void store_one(uint16_t* p, int e) const {
    *p = static_cast<uint16_t>((e < 2 ? w.x : w.y) >> ((e & 1) * 16));
  }
};

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

// Four logits from id v on (v may be negative or pass the row's end: `live` bits), their biases and mask bits.
struct Four {
  float x[4], b[4];
  uint32_t live, ok;   // bits of the ids that exist, and that the mask allows
};

template <typename TL>
struct Row {
  const TL* src;
  const float* bias;
  const uint32_t* mask;
  int V, turn;   // turn: how far an aligned bias vector begins before the ids' vector

  __device__ __forceinline__ void load(int v, Four& f) const {
    if (v >= 4 && v + 8 <= V) {   // the bias vectors on both sides lie within the row too
      load4(src + v, f.x);
      f.live = 15u;
      f.ok = 15u;
      if (mask) f.ok = __funnelshift_r(__ldg(mask + (v >> 5)), __ldg(mask + ((v + 3) >> 5)), v & 31) & 15u;
      if (bias) {
        const float4* p = reinterpret_cast<const float4*>(bias + v - turn);
        const float4 lo = __ldg(p);
        if (turn == 0) {
          f.b[0] = lo.x; f.b[1] = lo.y; f.b[2] = lo.z; f.b[3] = lo.w;
        } else {
          const float4 hi = __ldg(p + 1);
          f.b[0] = turn == 1 ? lo.y : (turn == 2 ? lo.z : lo.w);
          f.b[1] = turn == 1 ? lo.z : (turn == 2 ? lo.w : hi.x);
          f.b[2] = turn == 1 ? lo.w : (turn == 2 ? hi.x : hi.y);
          f.b[3] = turn == 1 ? hi.x : (turn == 2 ? hi.y : hi.z);
        }
      }
    } else {
      f.live = f.ok = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int id = v + e;
        f.x[e] = f.b[e] = 0.f;
        if (id >= 0 && id < V) {
          f.live |= 1u << e;
          if (!mask || ((__ldg(mask + (id >> 5)) >> (id & 31)) & 1u)) f.ok |= 1u << e;
          f.x[e] = as_float(src[id]);
          if (bias) f.b[e] = __ldg(bias + id);
        }
      }
    }
  }
};

template <typename TL>
__global__ void __launch_bounds__(kThreads, 4) adjust_kernel(AdjustArgs a) {
  extern __shared__ __align__(16) uint32_t counts[];   // 16-bit counters, four a vector; behind them the list
  __shared__ int listed;
  __shared__ float best_v[kWarps];
  __shared__ uint32_t best_i[kWarps];
  __shared__ unsigned long long part[kMaxSplit];
  uint16_t* list = reinterpret_cast<uint16_t*>(counts + 2 * a.at_once);   // counters that are not zero
  const int rank = blockIdx.x % a.split, row = blockIdx.x / a.split;   // row = t * N + n
  const int t = row / a.N, n = row - t * a.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long base = static_cast<long long>(row) * a.V;
  Row<TL> r;
  r.src = static_cast<const TL*>(a.logits) + base;
  r.bias = a.bias ? a.bias + static_cast<size_t>(n) * a.V : nullptr;
  r.mask = a.mask ? a.mask + static_cast<size_t>(row) * ((a.V + 31) / 32) : nullptr;
  r.V = a.V;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(r.src) / sizeof(TL)) & 3;
  r.turn = static_cast<int>(reinterpret_cast<uintptr_t>(r.bias) / 4 - shift) & 3;
  TL* dst = static_cast<TL*>(a.out) + base;
  const bool counted = a.history != nullptr;
  const int32_t* hist = counted ? a.history + static_cast<size_t>(t) * a.L * a.N + n : nullptr;
  // this CTA's vectors
  const int vecs = (a.V + shift + 3) / 4, per = (vecs + a.split - 1) / a.split;
  const int i_begin = rank * per, i_end = i_begin + per < vecs ? i_begin + per : vecs;
  // all that the first counts and vectors need is asked for at once
  int32_t early[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = static_cast<int>(threadIdx.x) + u * kThreads;
    early[u] = counted && i < a.L ? __ldg(hist + static_cast<size_t>(i) * a.N) : -1;
  }
  int len = 0;
  if (counted) {
    len = a.hist_lens ? __ldg(a.hist_lens + t) : a.L;
    len = len < 0 ? 0 : (len > a.L ? a.L : len);
  }
  const float rep = a.repetition ? __ldg(a.repetition + t) : 1.f, pre = a.presence ? __ldg(a.presence + t) : 0.f,
              frq = a.frequency ? __ldg(a.frequency + t) : 0.f;
  Four f[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int i = i_begin + static_cast<int>(threadIdx.x) + u * kThreads;
    if (i < i_end) r.load(4 * i - shift, f[u]);
  }
  float bv = __int_as_float(0xff800000);   // the best of this thread so far
  uint32_t bi = 0xFFFFFFFFu, low = 0xFFFFFFFFu;   // its id; the lowest id that may win at all
  for (int c0 = i_begin; c0 < i_end; c0 += a.at_once) {
    const int c1 = i_end - c0 < a.at_once ? i_end : c0 + a.at_once;
    const int first = 4 * c0 - shift;   // the id of counter 0
    // the id of a listed counter, what is known of it, and what becomes of it
    float lx = 0.f, lb = 0.f;
    bool lok = true;
    auto ask = [&](int id) {
      lx = as_float(r.src[id]);
      if (r.bias) lb = __ldg(r.bias + id);
      if (r.mask) lok = (__ldg(r.mask + (id >> 5)) >> (id & 31)) & 1u;
    };
    auto settle = [&](int at) {
      const uint32_t c = (counts[at >> 1] >> ((at & 1) * 16)) & 0xFFFFu;
      float x[4] = {lx, 0.f, 0.f, 0.f};
      if (a.repetition) x[0] = x[0] > 0.f ? __fdiv_rn(x[0], rep) : __fmul_rn(x[0], rep);
      if (a.frequency) x[0] = __fsub_rn(x[0], __fmul_rn(frq, static_cast<float>(c)));
      if (a.presence) x[0] = __fsub_rn(x[0], pre);
      if (r.bias) x[0] = __fadd_rn(x[0], lb);
      if (!lok) x[0] = __int_as_float(0xff800000);
      Out4<TL> o;
      o.round(x);
      o.store_one(dst + first + at, 0);
      if (lok && x[0] == x[0]) take(bv, bi, x[0], static_cast<uint32_t>(first + at));
    };
    int mine = -1;
    if (counted) {
      __syncthreads();   // the previous chunk's counts are read
      for (int i = threadIdx.x; i < c1 - c0; i += kThreads) reinterpret_cast<uint2*>(counts)[i] = make_uint2(0u, 0u);
      if (threadIdx.x == 0) listed = 0;
      __syncthreads();
      auto count = [&](int32_t id) {
        const unsigned at = static_cast<unsigned>(id - first);
        if (id >= 0 && id < a.V && at < 4u * (c1 - c0)) {
          const uint32_t was = atomicAdd(&counts[at >> 1], 1u << ((at & 1) * 16));
          if (((was >> ((at & 1) * 16)) & 0xFFFFu) == 0) list[atomicAdd(&listed, 1)] = static_cast<uint16_t>(at);
        }
        if (id >= a.V && rank == 0 && c0 == 0) record_device_error(a.errors);   // a negative id is no id
      };
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (static_cast<int>(threadIdx.x) + u * kThreads < len) count(early[u]);
#pragma unroll 4
      for (int i = threadIdx.x + 2 * kThreads; i < len; i += kThreads) count(__ldg(hist + static_cast<size_t>(i) * a.N));
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < listed) {
        mine = list[threadIdx.x];
        ask(first + mine);
      }
    }
    for (int at = c0; at < c1; at += kAhead * kThreads) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = at + static_cast<int>(threadIdx.x) + u * kThreads, v = 4 * i - shift;
        if (i >= c1) continue;
        uint32_t live = f[u].live, ok = f[u].ok;
        if (counted) {
          const uint2 c = reinterpret_cast<const uint2*>(counts)[i - c0];
          if (c.x | c.y) {
            const uint32_t rest = ((c.x & 0xFFFFu) == 0 ? 1u : 0u) | (c.x < 0x10000u ? 2u : 0u) |
                                  ((c.y & 0xFFFFu) == 0 ? 4u : 0u) | (c.y < 0x10000u ? 8u : 0u);
            live &= rest;
            ok &= rest;
          }
        }
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = r.bias ? __fadd_rn(f[u].x[e], f[u].b[e]) : f[u].x[e];
          if (!((ok >> e) & 1u)) x[e] = __int_as_float(0xff800000);
        }
        Out4<TL> o;
        o.round(x);
        if (live == 15u && a.same) {
          o.store(dst + v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((live >> e) & 1u) o.store_one(dst + v + e, e);
        }
        // Ids ascend along a thread's way, so only a larger value replaces its best one; NaN never does, nor does
        // the -inf of an id that is left out.  An allowed -inf counts when nothing larger comes.
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x[e] > bv) {
            bv = x[e];
            bi = static_cast<uint32_t>(v + e);
          }
        if (low == 0xFFFFFFFFu && ok) {
#pragma unroll
          for (int e = 3; e >= 0; --e)
            if (((ok >> e) & 1u) && x[e] == x[e]) low = static_cast<uint32_t>(v + e);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {   // the next vectors, of the next chunk too
        const int i = (at + kAhead * kThreads < c1 ? at + kAhead * kThreads : c1) + static_cast<int>(threadIdx.x) + u * kThreads;
        if (i < i_end) r.load(4 * i - shift, f[u]);
      }
    }
    if (mine >= 0) {
      settle(mine);
      for (int i = threadIdx.x + kThreads; i < listed; i += kThreads) {
        ask(first + list[i]);
        settle(list[i]);
      }
    }
  }
  if (!a.ids) return;   // uniform over the grid
  take(bv, bi, __int_as_float(0xff800000), low);
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
                                               kChunk * 4) != cudaSuccess)
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
  const int low = dtype == ZMOE_BF16 ? 7 : 15;   // a vector's bytes less one
  a.same = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(out)) & low) == 0;
  // enough CTAs for the machine, but at least 2048 ids each
  int split = 1;
  while (split < kMaxSplit && rows * split < 8LL * num_sms() && V / (2 * split) >= 2048) split *= 2;
  a.split = split;
  const int vecs = ((V + 6) / 4 + split - 1) / split;
  a.at_once = vecs < kChunk / 4 ? vecs : kChunk / 4;
  const int most = L < 4 * a.at_once ? L : 4 * a.at_once;   // ids that can be listed
  const size_t smem = a.history ? static_cast<size_t>(a.at_once) * 8 + static_cast<size_t>(most) * 2 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == ZMOE_BF16 ? launch<uint16_t>(a, static_cast<int>(rows), smem, s)
                            : launch<float>(a, static_cast<int>(rows), smem, s);
}
