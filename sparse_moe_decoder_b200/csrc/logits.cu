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
// (16-bit counters, as many ids at a time as fit), passes over its logits once, and leaves its best (value, id) in
// the first CTA's shared memory, which takes the largest: no workspace, one launch, and the order in which CTAs
// finish does not matter.
//
// The pass takes a vector of 16 bytes at an aligned address a thread at a time, two such vectors in flight; the
// first ones are on their way before the counting starts.  Rows of odd length start anywhere in a vector, so a
// vector's ids begin at E i - shift and the counters are laid out by id + shift; the ids of a row's first and last
// vectors go one by one, so nothing outside the row is touched.  How the bias lies against the logits is the same for
// a whole row, and the pass is compiled for each of the four ways (choosing the biases by it in the loop took three
// instructions an id).
//
// The pass leaves out the ids that were counted.  Few as they are, most warps hold one of them, and would take
// every step of the penalties for it; instead each is listed when its count leaves zero, as the ids at the ends are,
// and a thread of its own takes it.
//
// Measured: 9 x 1025, 128 frames: 3.9 us a call; 576 rows of 1025 with 512 frames and masks: 7.0 us; 192 x 100003 bf16
// with 2048 entries and masks: 45 us.  The pass alone takes 21.6 of them (its bytes at the copy rate 11.7, torch's copy of
// these rows 18.6), with biases and masks 30.7, with the counting and settling and neither 37.1 (102 us with the penalties
// within the pass).
#include <type_traits>

#include "sm100_ptx.cuh"
#include "vectors.cuh"

namespace zmoe {
namespace {

using namespace ptx;

constexpr int kAhead = 2;           // vectors in flight a thread
constexpr int kBlocks = 3;         // CTAs an SM, of 256 threads
constexpr int kMaxSplit = 8;       // the portable cluster size
constexpr int kEnds = 32;          // ids at a row's two ends, at most 4 + 7 and 4 + 2 * 7
constexpr int kEndVecs = 8;        // their vectors, rounded up
constexpr int kMaxSmem = 224 * 1024;
constexpr int kOneByOne = 4;
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
  int at_once;                // vectors counted at a time, beside those of the ends
  int list;                   // ids that can be listed, even
  int in_place;               // out is logits
  int same;                   // logits and out lie alike within a vector
  unsigned int* errors;
};

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(uint16_t v) { return bf16_to_f32(v); }
// A vector of 16 bytes: kE<TL> logits.  Plain loads: `out` may be `logits`.
template <typename TL>
constexpr int kE = 16 / sizeof(TL);

template <typename TL>
struct Vec;
template <>
struct Vec<float> {
  float4 w;
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* v) const { v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w; }
  __device__ __forceinline__ void round(const float* v) { w = make_float4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = w; }
};
template <>
struct Vec<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    widen_bf16x2(w.x, v);
    widen_bf16x2(w.y, v + 2);
    widen_bf16x2(w.z, v + 4);
    widen_bf16x2(w.w, v + 6);
  }
  __device__ __forceinline__ void round(const float* v) {
    w = make_uint4(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]), round_bf16x2(v[4], v[5]), round_bf16x2(v[6], v[7]));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = w; }
};
// Of a value that is rounded already.
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = static_cast<uint16_t>(__float_as_uint(v) >> 16); }
__device__ __forceinline__ float rounded(float, float v) { return v; }
__device__ __forceinline__ float rounded(uint16_t, float v) { return bf16_to_f32(f32_to_bf16_bits(v)); }

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

// The logits of a vector, their biases and mask bits.
template <typename TL>
struct Some {
  Vec<TL> x;
  float b[kE<TL>];
  uint32_t ok;   // bits of the ids that the mask allows
};

template <typename TL>
struct Row {
  const TL* src;
  const float* bias;
  const uint32_t* mask;

  // The vector from id v on; the bias vectors that overlap it lie within the row.  TURN: how far an aligned bias
  // vector begins before it (-1: no bias, kOneByOne: its biases one by one).
  template <int TURN>
  __device__ __forceinline__ void load(int v, Some<TL>& f) const {
    constexpr int E = kE<TL>;
    f.x.load(src + v);
    f.ok = (1u << E) - 1;
    if (mask) f.ok &= __funnelshift_r(mask[v >> 5], mask[(v + E - 1) >> 5], v & 31);
    if (TURN == kOneByOne) {
#pragma unroll
      for (int e = 0; e < E; ++e) f.b[e] = bias[v + e];
    } else if (TURN >= 0) {
      const float4* p = reinterpret_cast<const float4*>(bias + v - TURN);
      float w[E + 4];
#pragma unroll
      for (int i = 0; i < (TURN ? E / 4 + 1 : E / 4); ++i) {   // one more when they lie apart
        const float4 q = p[i];
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) f.b[e] = w[e + (TURN > 0 ? TURN & 3 : 0)];
    }
  }
};

template <typename TL, int kThreads>
__global__ void __launch_bounds__(kThreads, kBlocks * 256 / kThreads) adjust_kernel(AdjustArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t counts[];   // 16-bit counters, one an id; behind them the list
  __shared__ int listed;
  __shared__ float best_v[kWarps];
  __shared__ uint32_t best_i[kWarps];
  __shared__ unsigned long long part[kMaxSplit];
  // a bit for each counter that is not zero; listed ids, as counters, and their logits
  uint32_t* seen = counts + kE<TL> / 2 * (a.at_once + kEndVecs);
  uint16_t* list_at = reinterpret_cast<uint16_t*>(a.history ? seen + ((a.at_once + kEndVecs) * kE<TL> + 31) / 32 : counts);
  float* list_x = reinterpret_cast<float*>(list_at + a.list);
  enter_behind();
  const int rank = blockIdx.x % a.split, row = blockIdx.x / a.split;   // row = t * N + n
  const int t = row / a.N, n = row - t * a.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long base = static_cast<long long>(row) * a.V;
  Row<TL> r;
  r.src = static_cast<const TL*>(a.logits) + base;
  r.bias = a.bias ? a.bias + static_cast<size_t>(n) * a.V : nullptr;
  r.mask = a.mask ? a.mask + static_cast<size_t>(row) * ((a.V + 31) / 32) : nullptr;
  constexpr int E = kE<TL>;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(r.src) / sizeof(TL)) & (E - 1);
  const int turn = r.bias ? static_cast<int>(reinterpret_cast<uintptr_t>(r.bias) / 4 - shift) & 3 : -1;
  TL* dst = static_cast<TL*>(a.out) + base;
  const bool counted = a.history != nullptr;
  const int32_t* hist = counted ? a.history + static_cast<size_t>(t) * a.L * a.N + n : nullptr;
  // this CTA's vectors
  const int vecs = (a.V + shift + E - 1) / E, per = (vecs + a.split - 1) / a.split;
  const int i_begin = rank * per, i_end = i_begin + per < vecs ? i_begin + per : vecs;
  // the ids [0, low_end) and [high_begin, V) of the row go one by one, the vectors between them whole
  const int i_low = (4 + shift + E - 1) / E, i_high = a.V + shift >= E + 4 ? (a.V + shift - 4) / E : 0;
  const int low_end = E * i_low - shift < a.V ? E * i_low - shift : a.V;
  const int high_begin = E * i_high - shift > low_end ? E * i_high - shift : low_end;
  const int i_first = i_begin > i_low ? i_begin : i_low, i_last = i_end < i_high ? i_end : i_high;
  // the row's share (its first 256 KB: the CTAs' together fit the L2 cache) is on its way while the ids are counted
  if (threadIdx.x == 0 && i_last - i_first > kAhead * kThreads)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(r.src + (E * i_first - shift)),
                 "r"((i_last - i_first < 16384 ? i_last - i_first : 16384) * 16));
  // all that the first counts and vectors need is asked for at once
  int32_t early[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = static_cast<int>(threadIdx.x) + u * kThreads;
    early[u] = counted && i < a.L ? hist[static_cast<size_t>(i) * a.N] : -1;
  }
  int len = 0;
  if (counted) {
    len = a.hist_lens ? a.hist_lens[t] : a.L;
    len = len < 0 ? 0 : (len > a.L ? a.L : len);
  }
  const float rep = a.repetition ? a.repetition[t] : 1.f, pre = a.presence ? a.presence[t] : 0.f,
              frq = a.frequency ? a.frequency[t] : 0.f;
  const float none = __int_as_float(0xff800000);
  float bv = none;             // the best of this thread so far
  uint32_t bi = 0xFFFFFFFFu;   // its id
  auto pass = [&](auto turn_c) {
    constexpr int TURN = decltype(turn_c)::value;
    // This thread's vectors are kThreads apart from i_first on; its next kAhead are on their way at any time.
    constexpr int kStep = kAhead * kThreads;
    Some<TL> f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i_first + static_cast<int>(threadIdx.x) + u * kThreads;
      if (i < i_last) r.template load<TURN>(E * i - shift, f[u]);
    }
    // a chunk: `at_once` vectors (a multiple of kStep), and the ends of the row with the first and the last
    for (int s0 = i_first; s0 == i_first ? i_begin < i_end : s0 < i_last; s0 += a.at_once) {
      const int s1 = i_last - s0 < a.at_once ? i_last : s0 + a.at_once;
      const int c0 = s0 == i_first ? i_begin : s0, c1 = s1 >= i_last ? i_end : s1;
      const int first = E * c0 - shift;   // the id of counter 0
      const unsigned span = static_cast<unsigned>(E * (c1 - c0));
      __syncthreads();   // the previous chunk's counts and list are read
      if (counted) {
        for (int i = threadIdx.x; i < (c1 - c0) * E / 4; i += kThreads)
          reinterpret_cast<uint2*>(counts)[i] = make_uint2(0u, 0u);
        for (int i = threadIdx.x; i < ((c1 - c0) * E + 31) / 32; i += kThreads) seen[i] = 0u;
      }
      if (threadIdx.x == 0) listed = 0;
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < low_end + a.V - high_begin) {
        const int id = static_cast<int>(threadIdx.x) < low_end ? threadIdx.x : high_begin + threadIdx.x - low_end;
        const unsigned at = static_cast<unsigned>(id - first);
        if (at < span) list_at[atomicAdd(&listed, 1)] = static_cast<uint16_t>(at);
      }
      if (counted) {
        auto count = [&](int32_t id) {
          const unsigned at = static_cast<unsigned>(id - first);
          if (id >= 0 && at < span && id < a.V) {
            const uint32_t was = atomicAdd(&counts[at >> 1], 1u << ((at & 1) * 16));
            if (((was >> ((at & 1) * 16)) & 0xFFFFu) == 0 && id >= low_end && id < high_begin) {
              atomicOr(&seen[at >> 5], 1u << (at & 31));
              list_at[atomicAdd(&listed, 1)] = static_cast<uint16_t>(at);
            }
          }
          if (id >= a.V && rank == 0 && c0 == 0) record_device_error(a.errors);   // a negative id is no id
        };
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (static_cast<int>(threadIdx.x) + u * kThreads < len) count(early[u]);
#pragma unroll 4
        for (int i = threadIdx.x + 2 * kThreads; i < len; i += kThreads) count(hist[static_cast<size_t>(i) * a.N]);
      }
      __syncthreads();
      const int n_listed = listed;
      float lx = 0.f, lb = 0.f;
      bool lok = true;
      auto ask = [&](int i) {   // the logit, the bias and the mask of a listed id
        const int id = first + list_at[i];
        if (!a.in_place) lx = as_float(r.src[id]);
        if (TURN >= 0) lb = r.bias[id];
        if (r.mask) lok = (r.mask[id >> 5] >> (id & 31)) & 1u;
      };
      if (static_cast<int>(threadIdx.x) < n_listed) ask(threadIdx.x);
      if (a.in_place && n_listed) {   // read before the pass writes anything
#pragma unroll 4
        for (int i = threadIdx.x; i < n_listed; i += kThreads) list_x[i] = as_float(r.src[first + list_at[i]]);
        __syncthreads();
      }
      int best_at = -1, allowed_at = -1;   // the vector of this chunk's best, and the first that allows an id
      Vec<TL> best;
      auto rest_of = [&](int i) -> uint32_t {   // bits of the vector's ids that are not listed
        return ~(seen[(i - c0) * E >> 5] >> ((i - c0) * E & 31)) & ((1u << E) - 1);
      };
      for (int at = s0; at < s1; at += kStep) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int i = at + static_cast<int>(threadIdx.x) + u * kThreads, v = E * i - shift;
          if (i >= s1) continue;
          uint32_t ok = f[u].ok;
          if (counted) ok &= rest_of(i);
          float x[E];
          f[u].x.get(x);
          if (TURN >= 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __fadd_rn(x[e], f[u].b[e]);
          }
          if (ok != (1u << E) - 1) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (!((ok >> e) & 1u)) x[e] = none;
          }
          Vec<TL> o;
          o.round(x);
          // listed ids get their value behind the pass
          if (a.same) {
            o.store(dst + v);
          } else {
            o.get(x);
#pragma unroll
            for (int e = 0; e < E; ++e) store1(dst + v + e, x[e]);
          }
          // Vectors ascend along a thread's way, so only a larger value replaces the best one; NaN never does, nor
          // does the -inf of an id that is left out.  Rounding keeps the order.
          float top = x[0];
#pragma unroll
          for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
          top = rounded(TL(), top);
          if (top > bv) {
            bv = top;
            best_at = i;
            best = o;
          }
          if (allowed_at < 0 && ok) allowed_at = i;
          if (i + kStep < i_last) r.template load<TURN>(v + E * kStep, f[u]);   // of the next chunk too
        }
      }
      if (best_at >= 0) {
        float x[E];
        best.get(x);
#pragma unroll
        for (int e = E - 1; e >= 0; --e)
          if (x[e] == bv) bi = static_cast<uint32_t>(E * best_at - shift + e);
      } else if (bi == 0xFFFFFFFFu && allowed_at >= 0) {   // all that is allowed here is -inf or NaN: the first -inf
        for (int i = allowed_at; i < s1 && bi == 0xFFFFFFFFu; i += kThreads) {
          const int v = E * i - shift;
          uint32_t ok = counted ? rest_of(i) : (1u << E) - 1;
          if (r.mask) ok &= __funnelshift_r(r.mask[v >> 5], r.mask[(v + E - 1) >> 5], v & 31);
          for (int e = E - 1; e >= 0; --e)
            if (((ok >> e) & 1u) && as_float(dst[v + e]) == none) bi = static_cast<uint32_t>(v + e);
        }
      }
      if (n_listed) __syncthreads();   // the pass's vectors are written
      for (int i = threadIdx.x; i < n_listed; i += kThreads) {
        if (i >= kThreads) ask(i);
        const int at = list_at[i], id = first + at;
        const uint32_t c = counted ? (counts[at >> 1] >> ((at & 1) * 16)) & 0xFFFFu : 0u;
        float x = a.in_place ? list_x[i] : lx;
        if (c) {
          if (a.repetition) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
          if (a.frequency) x = __fsub_rn(x, __fmul_rn(frq, static_cast<float>(c)));
          if (a.presence) x = __fsub_rn(x, pre);
        }
        if (TURN >= 0) x = __fadd_rn(x, lb);
        x = lok ? rounded(TL(), x) : none;
        store1(dst + id, x);
        if (lok && x == x) take(bv, bi, x, static_cast<uint32_t>(id));
      }
    }
  };
  // The rows of a CTA's neighbours lie otherwise.  A short row's time goes into fetching the code, which they share
  // when there is one for all (576 rows of 1025: 9.4 to 7.0 us).
  if constexpr (kThreads == 128) {
    if (r.bias) pass(std::integral_constant<int, kOneByOne>());
    else pass(std::integral_constant<int, -1>());
  } else {
    switch (turn) {
      case -1: pass(std::integral_constant<int, -1>()); break;
      case 0: pass(std::integral_constant<int, 0>()); break;
      case 1: pass(std::integral_constant<int, 1>()); break;
      case 2: pass(std::integral_constant<int, 2>()); break;
      default: pass(std::integral_constant<int, 3>()); break;
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

template <typename TL, int kThreads>
zmoe_status launch(const AdjustArgs& a, int rows, size_t smem, cudaStream_t s) {
  if (smem > 40 * 1024 && cudaFuncSetAttribute(adjust_kernel<TL, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxSmem) != cudaSuccess)
    return check_launch("zmoe_adjust_logits: shared memory attribute");
  return launch_behind("zmoe_adjust_logits", adjust_kernel<TL, kThreads>, dim3(static_cast<unsigned>(rows) * a.split),
                       dim3(kThreads), smem, s, a.split, a);
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
  a.in_place = out == logits;
  a.same = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  // as many CTAs as run at once, with at least 2048 ids each
  int split = 1;
  while (split < kMaxSplit && rows * split * 2 <= static_cast<long long>(kBlocks) * num_sms() && V / (2 * split) >= 2048)
    split *= 2;
  a.split = split;
  const int E = dtype == ZMOE_BF16 ? 8 : 4;
  const int vecs = ((V + 2 * E - 2) / E + split - 1) / split;
  // Short rows take smaller CTAs, so that more of them run at once: always up to 512 vectors (576 rows of 1025 f32 with
  // biases and penalties: 6.9 us against 9.8), up to 1024 where not all rows run at once anyway (1809 rows of 4039 f32: 20.7
  // against 28.6, but 270 of them 8.9 against 7.3; one row of 6000: 5.8 against 5.3; 512 rows of 12000 bf16: 20.4 against
  // 16.7).
  const int threads = vecs <= 512 || (vecs <= 1024 && rows * split > static_cast<long long>(kBlocks) * num_sms()) ? 128 : 256;
  // As few chunks as fit shared memory beside the other CTAs of an SM (each takes the history anew) and a list of 16 bits.
  const int step = kAhead * threads;
  const long long ctas = rows * split;
  const int per_sm = ctas > 2LL * num_sms() ? 3 : (ctas > num_sms() ? 2 : 1);
  size_t smem = 0;
  for (int chunks = 1;; ++chunks) {
    a.at_once = ((vecs + chunks - 1) / chunks + step - 1) / step * step;
    const int counters = E * (a.at_once + kEndVecs);
    a.list = kEnds;
    if (a.history) {
      a.list += ((L < counters ? L : counters) + 1) & ~1;
      smem = static_cast<size_t>(counters) * 2 + (counters + 31) / 32 * 4 + static_cast<size_t>(a.list) * (a.in_place ? 6 : 2);
    } else {
      smem = static_cast<size_t>(a.list) * 6;
    }
    // a listed id is its place in the chunk, in 16 bits: with a history or without, a chunk has no more places
    if (counters <= 65536 && (smem <= kMaxSmem / per_sm || a.at_once == step)) break;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(rows);
  if (threads == 128)
    return dtype == ZMOE_BF16 ? launch<uint16_t, 128>(a, n, smem, s) : launch<float, 128>(a, n, smem, s);
  return dtype == ZMOE_BF16 ? launch<uint16_t, 256>(a, n, smem, s) : launch<float, 256>(a, n, smem, s);
}
