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
// Bound by HBM for prompts, by latency for decode steps.  D / 16 lanes carry a head, 16 columns each (eight of each
// half of its pairs), so a head's sum of squares is a shuffle within its lanes and every access is 16 bytes.  A
// group of lanes has two heads in flight; the first are asked for before the positions, so a decode step waits for
// memory twice: for the inputs and indices, then for the page's id.
#include "vectors.cuh"

namespace zmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;      // tokens of one block
constexpr int kMaxHalf = 64;       // pairs of one head (D <= 128)
constexpr int kAhead = 2;          // heads in flight a group of lanes

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

template <typename TI, int D, bool FP8>
__global__ void __launch_bounds__(kThreads, 3) kv_append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 16;                 // lanes of a head
  constexpr int kGroups = kThreads / kLanes;     // heads at a time
  __shared__ __align__(16) float2 turn[kMaxTokens][kMaxHalf];   // (cos, sin)
  __shared__ long long slot[kMaxTokens];         // cache row of head 0: page * Hkv * page_size + row; -1: skip
  const int t0 = blockIdx.x * a.tokens;
  const int nt = a.T - t0 < a.tokens ? a.T - t0 : a.tokens;
  const int half = a.rot >> 1;
  const int q_heads = a.q ? a.Hq : 0, heads = q_heads + 2 * a.Hkv;
  const int l = threadIdx.x % kLanes;
  // An item is a head of a token; this lane has its columns c0 .. c0 + 7 and c1 .. c1 + 7.  The heads of the
  // queries, the keys and the values are numbered one after another.
  struct Item {
    int tt, hd;
    __device__ __forceinline__ void wrap(int heads) {
      while (hd >= heads) {
        hd -= heads;
        ++tt;
      }
    }
  };
  struct Cols {
    int kind, hh, c0, c1;   // kind: query, key, value; hh: the head of its kind
    bool turned;
  };
  auto cols_of = [&](const Item& it) {
    Cols x;
    x.kind = it.hd < q_heads ? 0 : (it.hd < q_heads + a.Hkv ? 1 : 2);
    x.hh = it.hd - (x.kind == 0 ? 0 : (x.kind == 1 ? q_heads : q_heads + a.Hkv));
    x.turned = x.kind < 2 && 16 * l < a.rot;
    const bool apart = x.turned && !a.interleaved;
    x.c0 = apart ? 8 * l : 16 * l;
    x.c1 = x.c0 + (apart ? half : 8);
    return x;
  };
  Raw8<TI> raw[kAhead][2];
  Item at[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    at[u] = Item{0, static_cast<int>(threadIdx.x) / kLanes + u * kGroups};
    at[u].wrap(heads);
  }
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (at[u].tt < nt) {
        const Cols x = cols_of(at[u]);
        const TI* src = static_cast<const TI*>(x.kind == 0 ? a.q : (x.kind == 1 ? a.k : a.v)) +
                        (t0 + at[u].tt) * (x.kind == 0 ? a.q_stride : (x.kind == 1 ? a.k_stride : a.v_stride)) + x.hh * D;
        raw[u][0].load(src + x.c0);
        raw[u][1].load(src + x.c1);
      }
    }
  };
  fetch();
  if (threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    const int s = a.seq ? __ldg(a.seq + t) : t, p = __ldg(a.pos + t);
    long long to = -1;
    if (s >= 0) {   // a negative sequence marks a padding token
      const bool ok = s < a.n_seqs && p >= 0 && p < static_cast<long long>(a.max_pages) * a.page_size;
      const int col = ok ? static_cast<int>(static_cast<unsigned>(p) / static_cast<unsigned>(a.page_size)) : 0;
      const int page = ok ? __ldg(a.page_table + static_cast<size_t>(s) * a.max_pages + col) : -1;
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
          static_cast<double>(__ldg(a.pos + t0 + t)) * __ldg(a.inv_freq + f) * 0.15915494309189533577;   // 1 / (2 pi)
      float sn, cs;
      sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cs);
      turn[t][f] = make_float2(cs, sn);
    }
  }
  __syncthreads();
  for (int left = nt * heads; left > 0; left -= kAhead * kGroups) {   // every lane takes every round: they shuffle
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int tt = at[u].tt;
      const Cols it = cols_of(at[u]);
      float x[16];
      raw[u][0].get(x);
      raw[u][1].get(x + 8);
      const long long to = tt < nt ? slot[tt] : -1;
      const float* gamma = it.kind == 0 ? a.q_gamma : (it.kind == 1 ? a.k_gamma : nullptr);
      if (a.q_gamma || a.k_gamma) {   // the whole warp
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (gamma) {
          const float inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4* gp = reinterpret_cast<const float4*>(gamma + (k ? it.c1 : it.c0));
            const float4 g0 = __ldg(gp), g1 = __ldg(gp + 1);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * k + e] = x[8 * k + e] * inv * g[e];
          }
        }
      }
      if (to < 0) continue;
      if (it.turned) {
        const float4* w = reinterpret_cast<const float4*>(&turn[tt][8 * l]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 cs = w[e >> 1];   // (cos, sin) of two pairs
          if (a.interleaved) {
            const float y0 = x[2 * e], z0 = x[2 * e + 1], y1 = x[2 * e + 2], z1 = x[2 * e + 3];
            x[2 * e] = y0 * cs.x - z0 * cs.y;
            x[2 * e + 1] = y0 * cs.y + z0 * cs.x;
            x[2 * e + 2] = y1 * cs.z - z1 * cs.w;
            x[2 * e + 3] = y1 * cs.w + z1 * cs.z;
          } else {
            const float y0 = x[e], z0 = x[8 + e], y1 = x[e + 1], z1 = x[9 + e];
            x[e] = y0 * cs.x - z0 * cs.y;
            x[8 + e] = y0 * cs.y + z0 * cs.x;
            x[e + 1] = y1 * cs.z - z1 * cs.w;
            x[9 + e] = y1 * cs.w + z1 * cs.z;
          }
        }
      }
      if (it.kind == 0) {
        uint16_t* dst = a.q_out + (static_cast<size_t>(t0 + tt) * a.Hq + it.hh) * D;
        store8(dst + it.c0, x);
        store8(dst + it.c1, x + 8);
      } else {
        const size_t row = static_cast<size_t>(to + static_cast<long long>(it.hh) * a.page_size) * D;
        void* cache = it.kind == 1 ? a.k_cache : a.v_cache;
        if (FP8) {
          const float rs = __frcp_rn(__ldg((it.kind == 1 ? a.k_scale : a.v_scale) + it.hh));
          uint8_t* dst = static_cast<uint8_t*>(cache) + row;
          *reinterpret_cast<uint2*>(dst + it.c0) = make_uint2(e4m3x4(x, rs), e4m3x4(x + 4, rs));
          *reinterpret_cast<uint2*>(dst + it.c1) = make_uint2(e4m3x4(x + 8, rs), e4m3x4(x + 12, rs));
        } else {
          store8(static_cast<uint16_t*>(cache) + row + it.c0, x);
          store8(static_cast<uint16_t*>(cache) + row + it.c1, x + 8);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      at[u].hd += kAhead * kGroups;
      at[u].wrap(heads);
    }
    fetch();
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
