// zmoe_kv_append: queries and keys normed and rotated by position, keys and values stored in a paged cache.
//
// ZONOS2 Technical Report digest, "method overview and architecture", item 5 (grouped-query attention with
// rotary positions); "Builds on" lists the rotary embedding and the query/key norms.  Per token t at position
// p of sequence s, per head of width D:
//   y = x / sqrt(mean_c x_c^2 + eps) * gamma        (queries and keys, when a gain is given)
//   (y_a, y_b) <- (y_a cos w - y_b sin w, y_a sin w + y_b cos w),  w = p inv_freq[i]
// for the pairs i < R / 2 of the first R columns, (a, b) = (i, i + R / 2) or, interleaved, (2 i, 2 i + 1).
// The key and the value go to row p % page_size of page page_table[s, p / page_size].
//
// The angle is reduced in 64 bits to a fraction of a turn (p inv_freq / 2 pi less its nearest whole number), so
// that a far position costs no accuracy; the sine and cosine of the fraction are fp32.  They are formed once
// per token and pair in shared memory and serve every head of the token.
//
// Bound by HBM for prompts, by latency for decode steps.  D / 16 lanes carry a head, 16 columns each (the two
// halves of its pairs), so a head's sum of squares is a shuffle within its lanes and every access is 16 bytes.
#include <cuda_fp8.h>

#include "common.cuh"

namespace zmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;      // tokens of one block
constexpr int kMaxHalf = 64;       // pairs of one head (D <= 128)

struct AppendArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // elements between tokens
  const int32_t* seq;     // or null: token t belongs to sequence t
  const int32_t* pos;
  const double* inv_freq; // [rot / 2]
  int rot, interleaved;
  const float *q_gamma, *k_gamma;
  float eps;
  int T, Hq, Hkv, n_seqs, n_pages, page_size, max_pages, tokens;
  uint16_t* q_out;
  void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t* page_table;
  unsigned int* errors;
};

__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v);
}

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// E4M3 codes of v * r (nearest, saturating), r = fp32(1 / scale).
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float* v, float r) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i], r), __fmul_rn(v[4 * i + 1], r)),
                                                __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i + 2], r), __fmul_rn(v[4 * i + 3], r)),
                                                __NV_SATFINITE, __NV_E4M3);
    w[i] = (a & 0xFFFFu) | (b << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <typename TI, int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 16;                 // lanes of a head
  __shared__ float2 turn[kMaxTokens][kMaxHalf];  // (cos, sin)
  __shared__ long long slot[kMaxTokens];         // cache row of head 0: page * Hkv * page_size + row; -1: skip
  const int t0 = blockIdx.x * a.tokens;
  const int nt = a.T - t0 < a.tokens ? a.T - t0 : a.tokens;
  const int half = a.rot >> 1;
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    const int s = a.seq ? a.seq[t] : t;
    long long at = -1;
    if (s >= 0) {   // a negative sequence marks a padding token
      const int p = a.pos[t];
      const bool ok = s < a.n_seqs && p >= 0 && p < static_cast<long long>(a.max_pages) * a.page_size;
      const int page = ok ? a.page_table[static_cast<size_t>(s) * a.max_pages + p / a.page_size] : -1;
      if (page >= 0 && page < a.n_pages)
        at = static_cast<long long>(page) * a.Hkv * a.page_size + p % a.page_size;
      else
        record_device_error(a.errors);
    }
    slot[threadIdx.x] = at;
  }
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const double turns = static_cast<double>(a.pos[t0 + t]) * a.inv_freq[f] * 0.15915494309189533577;   // 1 / (2 pi)
    float sn, cs;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cs);
    turn[t][f] = make_float2(cs, sn);
  }
  __syncthreads();
  const int heads = (a.q ? a.Hq : 0) + 2 * a.Hkv, q_heads = heads - 2 * a.Hkv;
  const int l = threadIdx.x % kLanes;
  const int items = nt * heads, rounds = (items + kThreads / kLanes - 1) / (kThreads / kLanes);
  for (int r = 0; r < rounds; ++r) {
    const int item = r * (kThreads / kLanes) + threadIdx.x / kLanes;
    const int tt = item / heads, hd = item - tt * heads;
    const bool live = item < items && slot[tt < nt ? tt : 0] >= 0;
    const int kind = hd < q_heads ? 0 : (hd < q_heads + a.Hkv ? 1 : 2);   // query, key, value
    const int hh = kind == 0 ? hd : (kind == 1 ? hd - q_heads : hd - q_heads - a.Hkv);
    // this lane's two vectors of 8 columns
    int c0 = 16 * l, c1 = 16 * l + 8;
    const bool turned = kind < 2 && 16 * l < a.rot;
    if (!a.interleaved && turned) {
      c0 = 8 * l;
      c1 = 8 * l + half;
    }
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
    if (live) {
      const TI* src = static_cast<const TI*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) +
                      static_cast<long long>(t0 + tt) * (kind == 0 ? a.q_stride : (kind == 1 ? a.k_stride : a.v_stride)) +
                      static_cast<size_t>(hh) * D;
      load8(src + c0, x);
      load8(src + c1, x + 8);
    }
    const float* gamma = kind == 0 ? a.q_gamma : (kind == 1 ? a.k_gamma : nullptr);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!live) continue;
    if (gamma) {
      const float inv = rsqrtf(ss / static_cast<float>(D) + a.eps);
      float g[16];
      load8(gamma + c0, g);
      load8(gamma + c1, g + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * g[e];
    }
    if (turned) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = turn[tt][8 * l + e];
          const float u = x[2 * e], z = x[2 * e + 1];
          x[2 * e] = u * w.x - z * w.y;
          x[2 * e + 1] = u * w.y + z * w.x;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = turn[tt][8 * l + e];
          const float u = x[e], z = x[8 + e];
          x[e] = u * w.x - z * w.y;
          x[8 + e] = u * w.y + z * w.x;
        }
      }
    }
    if (kind == 0) {
      uint16_t* dst = a.q_out + (static_cast<size_t>(t0 + tt) * a.Hq + hh) * D;
      store8_bf16(dst + c0, x);
      store8_bf16(dst + c1, x + 8);
    } else {
      const size_t at = static_cast<size_t>(slot[tt] + static_cast<long long>(hh) * a.page_size) * D;
      void* cache = kind == 1 ? a.k_cache : a.v_cache;
      if (FP8) {
        const float rs = __frcp_rn((kind == 1 ? a.k_scale : a.v_scale)[hh]);
        store8_e4m3(static_cast<uint8_t*>(cache) + at + c0, x, rs);
        store8_e4m3(static_cast<uint8_t*>(cache) + at + c1, x + 8, rs);
      } else {
        store8_bf16(static_cast<uint16_t*>(cache) + at + c0, x);
        store8_bf16(static_cast<uint16_t*>(cache) + at + c1, x + 8);
      }
    }
  }
}

template <typename TI>
void launch(const AppendArgs& a, int D, bool fp8, int grid, cudaStream_t s) {
  if (D == 64) {
    if (fp8) kv_append_kernel<TI, 64, true><<<grid, kThreads, 0, s>>>(a);
    else kv_append_kernel<TI, 64, false><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (fp8) kv_append_kernel<TI, 128, true><<<grid, kThreads, 0, s>>>(a);
    else kv_append_kernel<TI, 128, false><<<grid, kThreads, 0, s>>>(a);
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace zmoe

extern "C" zmoe_status zmoe_kv_append(const void* q, const void* k, const void* v, zmoe_dtype in_dtype,
                                      int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* seq,
                                      const int32_t* pos, const double* inv_freq, int rotary_dim, int interleaved,
                                      const float* q_gamma, const float* k_gamma, float eps, int T, int Hq, int Hkv,
                                      int D, void* q_out, void* k_cache, void* v_cache, zmoe_dtype kv_dtype,
                                      const float* k_scale, const float* v_scale, const int32_t* page_table,
                                      int n_seqs, int max_pages, int n_pages, int page_size, zmoe_stream_t stream) {
  ZMOE_TRACE("zmoe_kv_append");
  using namespace zmoe;
  ZMOE_REQUIRE(dtype_ok(in_dtype), "zmoe_kv_append: the inputs are f32 or bf16");
  ZMOE_REQUIRE(kv_dtype == ZMOE_BF16 || kv_dtype == ZMOE_E4M3, "zmoe_kv_append: the cache is bf16 or E4M3");
  ZMOE_REQUIRE(T >= 0 && Hkv >= 1 && Hq >= 0 && n_seqs >= 0, "zmoe_kv_append: bad T, Hq, Hkv or n_seqs");
  ZMOE_REQUIRE(D >= 1 && rotary_dim >= 0 && rotary_dim <= D && rotary_dim % 16 == 0,
               "zmoe_kv_append: rotary_dim must be a multiple of 16 up to D");
  ZMOE_REQUIRE(page_size >= 16 && page_size % 16 == 0, "zmoe_kv_append: page_size must be a multiple of 16");
  ZMOE_REQUIRE(max_pages >= 0 && n_pages >= 0, "zmoe_kv_append: bad max_pages or n_pages");
  ZMOE_REQUIRE(eps >= 0.f, "zmoe_kv_append: eps must be >= 0");
  ZMOE_REQUIRE(seq || T <= n_seqs, "zmoe_kv_append: without seq every token is a sequence of its own: T <= n_seqs");
  if (T == 0) return ZMOE_OK;
  ZMOE_REQUIRE(k && v && pos && k_cache && v_cache && page_table, "zmoe_kv_append: NULL pointer");
  ZMOE_REQUIRE((q != nullptr) == (q_out != nullptr) && (!q || Hq >= 1), "zmoe_kv_append: q and q_out come together");
  ZMOE_REQUIRE(rotary_dim == 0 || inv_freq, "zmoe_kv_append: rotary_dim > 0 needs inv_freq");
  ZMOE_REQUIRE(kv_dtype == ZMOE_BF16 || (k_scale && v_scale), "zmoe_kv_append: an E4M3 cache needs k_scale and v_scale");
  if (D != 64 && D != 128) return fail(ZMOE_ERR_UNSUPPORTED, "zmoe_kv_append: D must be 64 or 128");
  const long long step = in_dtype == ZMOE_BF16 ? 8 : 4;
  ZMOE_REQUIRE((!q || (q_stride >= static_cast<long long>(Hq) * D && q_stride % step == 0)) &&
                   k_stride >= static_cast<long long>(Hkv) * D && k_stride % step == 0 &&
                   v_stride >= static_cast<long long>(Hkv) * D && v_stride % step == 0,
               "zmoe_kv_append: a token's stride must hold its heads and be a multiple of 16 bytes");
  ZMOE_REQUIRE((!q || (aligned16(q) && aligned16(q_out))) && aligned16(k) && aligned16(v) && aligned16(k_cache) &&
                   aligned16(v_cache) && (!q_gamma || aligned16(q_gamma)) && (!k_gamma || aligned16(k_gamma)) &&
                   aligned(inv_freq, 8) && aligned(pos, 4) && aligned(seq, 4) && aligned(page_table, 4) &&
                   aligned(k_scale, 4) && aligned(v_scale, 4),
               "zmoe_kv_append: pointers must be 16-byte aligned");
  ZMOE_REQUIRE(static_cast<long long>(max_pages) * page_size <= 0x7fffffffLL,
               "zmoe_kv_append: max_pages * page_size overflows int32");
  ZMOE_REQUIRE(static_cast<long long>(Hq) + 2LL * Hkv <= 0xffffLL, "zmoe_kv_append: too many heads");
  clear_error();
  AppendArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.seq = seq; a.pos = pos; a.inv_freq = inv_freq;
  a.rot = rotary_dim; a.interleaved = interleaved;
  a.q_gamma = q_gamma; a.k_gamma = k_gamma; a.eps = eps;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.n_seqs = n_seqs; a.n_pages = n_pages; a.page_size = page_size;
  a.max_pages = max_pages;
  a.tokens = T > 4 * num_sms() ? kMaxTokens : 1;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.page_table = page_table;
  a.errors = device_error_counter();
  const int grid = (T + a.tokens - 1) / a.tokens;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (in_dtype == ZMOE_BF16) launch<uint16_t>(a, D, kv_dtype == ZMOE_E4M3, grid, s);
  else launch<float>(a, D, kv_dtype == ZMOE_E4M3, grid, s);
  return check_launch("zmoe_kv_append");
}
