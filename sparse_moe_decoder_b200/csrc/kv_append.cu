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
// Bound by HBM for prompts, by latency for decode steps.  D / 16 lanes carry a head, so its sum of squares is a
// shuffle within them.  A lane has two sets of 4 + 4 columns, four pairs each; neighbouring lanes have neighbouring
// fours, so that a load instruction reads whole lines (with eight neighbouring columns a lane the L1 cache was what
// bounded f32 prompts).  A head's values are asked for before the positions, so a decode step waits for memory twice:
// for the inputs and indices, then for the page's id.  One head in flight a group of lanes and four blocks an SM beat
// two heads and three blocks (55 against 62 us below); eight tokens a block share the angles.
//
// Measured: 16384 tokens, 16 query and 4 key heads of 128, f32 into bf16: 54.8 us, 5.5 TB/s, into E4M3 52 us, 5.5 TB/s;
// bf16 into either 45 us (4.4 and 4.1 TB/s); 2997 tokens, 12 + 2 heads of 64, bf16 into E4M3: 5.4 us, 2.1 TB/s; 64 tokens:
// 3.6 us a call.
#include "vectors.cuh"

namespace zmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;      // tokens of one block
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

// Four neighbouring values as they lie in memory, and as fp32.
template <typename TI>
struct Raw4;
template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* v) const { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
};
template <>
struct Raw4<uint16_t> {
  uint2 r;
  __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    widen_bf16x2(r.x, v);
    widen_bf16x2(r.y, v + 2);
  }
};

__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
}

template <typename TI, int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 4) kv_append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 16;                 // lanes of a head
  constexpr int kGroups = kThreads / kLanes;     // heads at a time
  __shared__ __align__(16) float cosine[kMaxTokens][kMaxHalf], sine[kMaxTokens][kMaxHalf];
  __shared__ long long slot[kMaxTokens];         // cache row of head 0: page * Hkv * page_size + row; -1: skip
  enter_behind();
  const int t0 = blockIdx.x * a.tokens;
  const int nt = a.T - t0 < a.tokens ? a.T - t0 : a.tokens;
  const int half = a.rot >> 1;
  const int q_heads = a.q ? a.Hq : 0, heads = q_heads + 2 * a.Hkv;
  const int l = threadIdx.x % kLanes;
  // An item is a head of a token.  The heads of the queries, the keys and the values are numbered one after another.
  struct Item {
    int tt, hd;
    __device__ __forceinline__ void wrap(int heads) {
      while (hd >= heads) {
        hd -= heads;
        ++tt;
      }
    }
  };
  // Set k of this lane's columns: c0 .. c0 + 3 and c1 .. c1 + 3.
  struct Cols {
    int c0, c1;
    bool turned;
  };
  Cols cols[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int j = l + k * kLanes;   // of the head's D / 8 sets, the turned ones first
    cols[k].turned = 8 * j < a.rot;
    if (a.interleaved) {
      cols[k].c0 = 8 * j;
      cols[k].c1 = 8 * j + 4;
    } else if (cols[k].turned) {
      cols[k].c0 = 4 * j;
      cols[k].c1 = half + 4 * j;
    } else {
      cols[k].c0 = half + 4 * j;   // rot + 4 (j - rot / 8)
      cols[k].c1 = cols[k].c0 + (D - a.rot) / 2;
    }
  }
  Raw4<TI> raw[4];
  Item at{0, static_cast<int>(threadIdx.x) / kLanes};
  at.wrap(heads);
  auto fetch = [&]() {
    if (at.tt < nt) {
      const int hd = at.hd;
      const TI* src = hd < q_heads ? static_cast<const TI*>(a.q) + (t0 + at.tt) * a.q_stride + hd * D
                      : hd < q_heads + a.Hkv
                          ? static_cast<const TI*>(a.k) + (t0 + at.tt) * a.k_stride + (hd - q_heads) * D
                          : static_cast<const TI*>(a.v) + (t0 + at.tt) * a.v_stride + (hd - q_heads - a.Hkv) * D;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        raw[2 * k].load(src + cols[k].c0);
        raw[2 * k + 1].load(src + cols[k].c1);
      }
    }
  };
  fetch();
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    const int s = a.seq ? a.seq[t] : t, p = a.pos[t];
    long long to = -1;
    if (s >= 0) {   // a negative sequence marks a padding token
      const bool ok = s < a.n_seqs && p >= 0 && p < static_cast<long long>(a.max_pages) * a.page_size;
      const int col = ok ? static_cast<int>(static_cast<unsigned>(p) / static_cast<unsigned>(a.page_size)) : 0;
      const int page = ok ? a.page_table[static_cast<size_t>(s) * a.max_pages + col] : -1;
      if (page >= 0 && page < a.n_pages)
        to = static_cast<long long>(page) * a.Hkv * a.page_size + (p - col * a.page_size);
      else
        record_device_error(a.errors);
    }
    slot[threadIdx.x] = to;
  }
  for (int i = threadIdx.x; i < kMaxTokens * kMaxHalf; i += kThreads) {
    const int t = i / kMaxHalf, f = i % kMaxHalf;
    if (t < nt && f < half) {
      const double turns =
          static_cast<double>(a.pos[t0 + t]) * a.inv_freq[f] * 0.15915494309189533577;   // 1 / (2 pi)
      float sn, cs;
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cs);
      cosine[t][f] = cs;
      sine[t][f] = sn;
    }
  }
  __syncthreads();
  for (int left = nt * heads; left > 0; left -= kGroups) {   // every lane takes every round: they shuffle
    const int tt = at.tt, hd = at.hd;
    float x[2][8];   // [set][columns c0 .., c1 ..]
#pragma unroll
    for (int k = 0; k < 4; ++k) raw[k].get(&x[k >> 1][4 * (k & 1)]);
    const long long to = tt < nt ? slot[tt] : -1;
    const float* gamma = hd < q_heads ? a.q_gamma : (hd < q_heads + a.Hkv ? a.k_gamma : nullptr);
    if (a.q_gamma || a.k_gamma) {   // the whole warp
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e >> 3][e & 7], x[e >> 3][e & 7], ss);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (gamma) {
        const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 g0 = *reinterpret_cast<const float4*>(gamma + cols[k].c0);
          const float4 g1 = *reinterpret_cast<const float4*>(gamma + cols[k].c1);
          const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = x[k][e] * inv * g[e];
        }
      }
    }
    if (to >= 0) {
      if (hd < q_heads + a.Hkv) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!cols[k].turned) continue;
          const float4 c4 = *reinterpret_cast<const float4*>(&cosine[tt][4 * (l + k * kLanes)]);
          const float4 s4 = *reinterpret_cast<const float4*>(&sine[tt][4 * (l + k * kLanes)]);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (a.interleaved) {
              const float y = x[k][2 * e], z = x[k][2 * e + 1];
              x[k][2 * e] = y * c[e] - z * s[e];
              x[k][2 * e + 1] = y * s[e] + z * c[e];
            } else {
              const float y = x[k][e], z = x[k][4 + e];
              x[k][e] = y * c[e] - z * s[e];
              x[k][4 + e] = y * s[e] + z * c[e];
            }
          }
        }
      }
      if (hd < q_heads) {
        uint16_t* dst = a.q_out + (static_cast<size_t>(t0 + tt) * a.Hq + hd) * D;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          store4(dst + cols[k].c0, x[k]);
          store4(dst + cols[k].c1, x[k] + 4);
        }
      } else {
        const bool key = hd < q_heads + a.Hkv;
        const int hh = hd - q_heads - (key ? 0 : a.Hkv);
        const size_t row = static_cast<size_t>(to + static_cast<long long>(hh) * a.page_size) * D;
        void* cache = key ? a.k_cache : a.v_cache;
        if (FP8) {
          const float rs = __frcp_rn((key ? a.k_scale : a.v_scale)[hh]);
          uint8_t* dst = static_cast<uint8_t*>(cache) + row;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            *reinterpret_cast<uint32_t*>(dst + cols[k].c0) = e4m3x4(x[k], rs);
            *reinterpret_cast<uint32_t*>(dst + cols[k].c1) = e4m3x4(x[k] + 4, rs);
          }
        } else {
          uint16_t* dst = static_cast<uint16_t*>(cache) + row;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            store4(dst + cols[k].c0, x[k]);
            store4(dst + cols[k].c1, x[k] + 4);
          }
        }
      }
    }
    at.hd += kGroups;
    at.wrap(heads);
    fetch();
  }
}

template <typename TI, int D>
zmoe_status launch(const AppendArgs& a, bool fp8, int grid, cudaStream_t s) {
  return launch_behind("zmoe_kv_append", fp8 ? kv_append_kernel<TI, D, true> : kv_append_kernel<TI, D, false>, dim3(grid),
                       dim3(kThreads), 0, s, 1, a);
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
  // tokens of a block: up to 8, as long as there are two blocks for each SM
  a.tokens = T / (2 * num_sms());
  a.tokens = a.tokens < 1 ? 1 : (a.tokens < kMaxTokens ? a.tokens : kMaxTokens);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.page_table = page_table;
  a.errors = device_error_counter();
  const int grid = (T + a.tokens - 1) / a.tokens;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = kv_dtype == ZMOE_E4M3;
  if (in_dtype == ZMOE_BF16) return D == 64 ? launch<uint16_t, 64>(a, fp8, grid, s) : launch<uint16_t, 128>(a, fp8, grid, s);
  return D == 64 ? launch<float, 64>(a, fp8, grid, s) : launch<float, 128>(a, fp8, grid, s);
}
