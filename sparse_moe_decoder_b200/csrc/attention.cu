// zmoe_paged_attention: attention of one new token per sequence over a paged key-value cache.
//
// ZONOS2 Technical Report digest, "method overview and architecture", item 5 (grouped-query attention with
// headwise gating).  Per sequence b with n = lens[b] cached tokens and query head i of key-value head g:
//   s_t = scale q_i . k_t;   o_i = sum_t exp(s_t) v_t / sum_t exp(s_t),  t < n;   lse_i = log sum_t exp(s_t)
//   out_i = sigmoid(gate_i) o_i                                               (o = 0, lse = -inf when n = 0)
//
// Bound by HBM: every cached key and value is read once (per 8 or 16 query heads of a group).  A warp takes 16
// tokens at a time, which lie in one page, straight into registers: no shared memory, no barrier in the loop.
//   scores  S = Q K^T:      m16n8k16, 16 rows of query heads (8 or 16 in use), 8 tokens, 16 columns;
//   output  O^T = V^T P^T:  m16n8k16, 16 columns of V, 8 query heads, 16 tokens.
// The contraction index of a tensor-core product may be permuted as long as both operands agree, so each lane's
// share of a key row is 16 contiguous bytes, and each lane's share of the output is D / 8 contiguous columns.
// S leaves the first product in the layout that the second takes P^T in.  The maximum and the sum of the
// softmax run along in registers.
//
// The loads of the next 16 keys are issued as soon as S is formed, those of the next values as soon as O is.
//
// Work is split over the cache's length: the (sequence, group, 16-token tile) triples are one line of tiles,
// cut into equal pieces, one a warp, so that ragged lengths balance.  A warp writes the groups that lie within
// its piece; of a group that is cut it leaves (maximum, sum, O) in the workspace, and a second kernel, launched
// to start early (programmatic dependent launch), joins them in a fixed order.
//
// P is split into two 16-bit terms, P = P_hi + P_lo (the second product runs twice): one bf16 term alone would
// cost 2^-9 of every weight.  An infinite value times a P_lo of zero or of the other sign would be NaN where the
// formula has an infinity, so a piece whose output holds a NaN is passed over once more with the second term
// leaving infinities out.  An 8-bit cache is expanded to f16, exactly; its queries are scaled by a power of
// two per head to use f16's range, and so is P.
#include "sm100_ptx.cuh"

namespace zmoe {
namespace {

using namespace ptx;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWarpsPerSm = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  const uint16_t* q;      // [B, Hq, D]
  const void *k, *v;      // [n_pages, Hkv, page_size, D]
  const float *k_scale, *v_scale;
  const int32_t* table;   // [B, max_pages]
  const int32_t* lens;    // [B]
  const float* gate;      // [B, Hq] or null
  float scale;
  int B, Hq, Hkv, G, gtiles, max_pages, n_pages, page_size;
  void* out;              // [B, Hq, D]
  float* lse;             // [B, Hq] or null
  float* parts;           // [warps][2] of {m[H], l[H], O[H][D]}, H = 8 HT
  int warps;              // warps of the first kernel
  unsigned int* errors;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Tiles of 16 tokens of sequence b; a length beyond the table's pages is an error and cut to them.
__device__ __forceinline__ int seq_len(const AttnArgs& a, int b) {
  const int n = __ldg(a.lens + b);
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  return n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
}

__device__ __forceinline__ int tiles_of(int n) { return static_cast<int>((static_cast<unsigned>(n) + 15u) >> 4); }

__device__ __forceinline__ long long divide(long long x, long long y) {   // of numbers that are not negative
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// `total` tiles in `count` pieces, one a warp, none empty: the first `more` pieces have one tile more.
struct Pieces {
  int count;
  long long size, more;

  __device__ __forceinline__ Pieces(long long total, int warps)
      : count(total < warps ? static_cast<int>(total) : warps), size(divide(total, count)), more(total - size * count) {}
  __device__ __forceinline__ long long start(long long w) const { return w * size + (w < more ? w : more); }
  __device__ __forceinline__ int owner(long long x) const {   // the warp whose piece tile x is in
    const long long big = more * (size + 1);
    return static_cast<int>(x < big ? divide(x, size + 1) : more + divide(x - big, size));
  }
};

// Exclusive prefix over the block's threads of `mine`; every thread receives the total.
__device__ __forceinline__ long long block_prefix(long long mine, long long* scratch, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  return before + inc - mine;
}

template <int D, int HT>
__host__ __device__ constexpr int part_floats() {
  return 8 * HT * (D + 2);
}

// The types of an 8-bit or a bf16 cache: 16-byte vectors of a lane per key row, and bytes of a lane per value row.
template <int D, bool FP8>
struct Lay {
  static constexpr int esz = FP8 ? 1 : 2;
  static constexpr int kvecs = D * esz / 64;       // 16-byte vectors of a key row per lane (4 lanes a row)
  static constexpr int vwords = D * esz / 32;      // 32-bit words of a value row per lane (8 lanes a row)
  static constexpr int steps = D / 16;             // 16-column steps of the first product
  static constexpr int mt = D / 16;                // 16-column tiles of the output
};

template <int D, bool FP8>
__device__ __forceinline__ void load_k(const unsigned char* rows, int g, int j, uint4 (&k)[2][Lay<D, FP8>::kvecs]) {
  using L = Lay<D, FP8>;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < L::kvecs; ++c)
      k[r][c] = ldg_stream(rows + static_cast<size_t>(g + 8 * r) * (D * L::esz) + c * 64 + j * 16);
}

template <int D, bool FP8>
__device__ __forceinline__ void load_v(const unsigned char* rows, int g, int j, uint32_t (&v)[4][Lay<D, FP8>::vwords]) {
  using L = Lay<D, FP8>;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int tok = 2 * j + (r & 1) + 8 * (r >> 1);
    const unsigned char* p = rows + static_cast<size_t>(tok) * (D * L::esz);
    if (L::vwords == 2) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + g * 8));
      v[r][0] = w.x;
      v[r][1] = w.y;
    } else {
#pragma unroll
      for (int c = 0; c < L::vwords / 4; ++c) {
        const uint4 w = ldg_stream(p + c * 128 + g * 16);
        v[r][4 * c] = w.x;
        v[r][4 * c + 1] = w.y;
        v[r][4 * c + 2] = w.z;
        v[r][4 * c + 3] = w.w;
      }
    }
  }
}

// Two bf16 values, infinities and NaN replaced by 0.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t x) {
  if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
  if ((x & 0x7F800000u) == 0x7F800000u) x &= 0x0000FFFFu;
  return x;
}

// The column of V that word w's lower half (bf16) or first byte (8 bits) of lane group g holds.
template <int D, bool FP8>
__device__ __forceinline__ int v_col(int g, int w) {
  if (FP8) return g * (D / 8) + 4 * w;
  return (w >> 2) * 64 + g * 8 + 2 * (w & 3);
}

template <typename TO>
__device__ __forceinline__ void store2(TO* p, float x, float y);
template <>
__device__ __forceinline__ void store2<float>(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
template <>
__device__ __forceinline__ void store2<uint16_t>(uint16_t* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}

__device__ __forceinline__ float gate_of(const AttnArgs& a, int b, int head) {
  return a.gate ? 1.f / (1.f + expf(-__ldg(a.gate + static_cast<size_t>(b) * a.Hq + head))) : 1.f;
}

template <int D, bool FP8, int HT, typename TO>
__global__ void __launch_bounds__(kThreads, HT == 1 ? 3 : 2) attn_kernel(AttnArgs a) {
  using L = Lay<D, FP8>;
  constexpr int H = 8 * HT;
  constexpr float kPScale = FP8 ? 32768.f : 1.f;   // f16 holds P in [0, 2^15]: weights down to 2^-39 survive
  __shared__ long long scan[kWarps];
  __shared__ int at_b[kWarps];
  __shared__ long long at_off[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  const int units = a.Hkv * a.gtiles;
  // the line of tiles: sequence by sequence, in each the groups, in each the tiles
  const int per = (a.B + kThreads - 1) / kThreads, b_lo = threadIdx.x * per;
  const int b_hi = b_lo + per < a.B ? b_lo + per : a.B;
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += static_cast<long long>(tiles_of(seq_len(a, b))) * units;
    if (blockIdx.x == 0 && __ldg(a.lens + b) > static_cast<long long>(a.max_pages) * a.page_size)
      record_device_error(a.errors);
  }
  long long total;
  const long long pre = block_prefix(mine, scan, total);
  if (total == 0) return;
  const Pieces pieces(total, a.warps);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long x = pieces.start(static_cast<long long>(blockIdx.x) * kWarps + w);
    if (x >= pre && x < pre + mine) {
      long long p = pre;
      int b = b_lo;
      for (;; ++b) {
        const long long n = static_cast<long long>(tiles_of(seq_len(a, b))) * units;
        if (x < p + n) break;
        p += n;
      }
      at_b[w] = b;
      at_off[w] = x - p;
    }
  }
  __syncthreads();
  const long long gw = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (gw >= pieces.count) return;
  const long long x0 = pieces.start(gw), x1 = pieces.start(gw + 1);
  int b = at_b[warp], n = seq_len(a, b), nt = tiles_of(n);
  int u = static_cast<int>(at_off[warp] / nt), tile = static_cast<int>(at_off[warp] - static_cast<long long>(u) * nt);
  const int tpp = a.page_size >> 4;   // tiles per page
  for (long long x = x0; x < x1;) {
    const int t_end = x1 - x < nt - tile ? tile + static_cast<int>(x1 - x) : nt;
    const int hk = u / a.gtiles, row0 = (u - hk * a.gtiles) * H;
    // queries of heads row0 + g (and + 8) of the group; rows beyond the group are zero
    uint32_t qf[L::steps][4];
    float qs[HT];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool on = r < HT && row0 + g + 8 * r < a.G;
      const uint16_t* qr =
          a.q + (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(hk) * a.G + (on ? row0 + g + 8 * r : 0)) * D;
      uint4 raw[D / 32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        // lane j's columns: 8 from 32 c + 8 j (bf16), 16 from 64 c' + 16 j (8-bit cache)
        const int col = FP8 ? (c >> 1) * 64 + j * 16 + (c & 1) * 8 : c * 32 + j * 8;
        raw[c] = on ? __ldg(reinterpret_cast<const uint4*>(qr + col)) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (r < HT) qs[r] = a.scale * kLog2e;
      if (FP8) {
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float f[8];
          unpack_bf16x8(raw[c], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest magnitude goes to [2^14, 2^15)
        const int ex = top > 0.f && top < __int_as_float(0x7f800000) ? 14 - ilogbf(top) : 0;
        if (r < HT) qs[r] = ldexpf(a.scale * kLog2e * __ldg(a.k_scale + hk), -ex);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float f[8];
          unpack_bf16x8(raw[c], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = ldexpf(f[e], ex);
          raw[c] = make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                              pack_f16x2(f[6], f[7]));
        }
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        qf[2 * c][r] = raw[c].x;
        qf[2 * c][2 + r] = raw[c].y;
        qf[2 * c + 1][r] = raw[c].z;
        qf[2 * c + 1][2 + r] = raw[c].w;
      }
    }
    float o[HT][L::mt][4];
    float m[HT], l[HT];
    bool careful = false;
  again:
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      m[h] = __int_as_float(0xff800000);
      l[h] = 0.f;
#pragma unroll
      for (int i = 0; i < L::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][i][e] = 0.f;
    }
    // cache row of tile t's first token, for the 32 tiles from `win` on (lane i: tile win + i); 0xffffffff: no page
    int win = tile;
    auto rows_of = [&](int t) -> uint32_t {
      uint32_t r = 0xFFFFFFFFu;
      if (t < t_end) {
        const int col = t / tpp;
        const int pid = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + col);
        if (pid >= 0 && pid < a.n_pages)
          r = (static_cast<uint32_t>(pid) * a.Hkv + hk) * a.page_size + static_cast<uint32_t>(t - col * tpp) * 16u;
        else if (u == 0 && (t == tile || t == col * tpp))
          record_device_error(a.errors);
      }
      return r;
    };
    uint32_t rows = rows_of(win + lane);
    auto row_at = [&](int t) { return __shfl_sync(0xffffffffu, rows, t - win); };
    const unsigned char* kbase = static_cast<const unsigned char*>(a.k);
    const unsigned char* vbase = static_cast<const unsigned char*>(a.v);
    uint4 kr[2][L::kvecs];
    uint32_t vr[4][L::vwords];
    uint32_t row = row_at(tile);
    bool have = row != 0xFFFFFFFFu;
    load_k<D, FP8>(kbase + static_cast<size_t>(have ? row : 0u) * (D * L::esz), g, j, kr);
    load_v<D, FP8>(vbase + static_cast<size_t>(have ? row : 0u) * (D * L::esz), g, j, vr);
    for (int t = tile; t < t_end; ++t) {
      const int left = have ? n - t * 16 : 0, live = left < 16 ? left : 16;   // tokens of this tile that count
      float s[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[r][e] = 0.f;
#pragma unroll
        for (int c = 0; c < L::kvecs; ++c) {
          const uint32_t w[4] = {kr[r][c].x, kr[r][c].y, kr[r][c].z, kr[r][c].w};
          if (FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16(s[r], qf[4 * c + i], e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] & 0xFFFFu)),
                      e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16)));
          } else {
            mma_bf16(s[r], qf[2 * c], w[0], w[1]);
            mma_bf16(s[r], qf[2 * c + 1], w[2], w[3]);
          }
        }
      }
      // the next keys
      bool next_have = false;
      uint32_t next_row = 0;
      if (t + 1 < t_end) {
        if (t + 1 - win == 32) {
          win = t + 1;
          rows = rows_of(win + lane);
        }
        next_row = row_at(t + 1);
        next_have = next_row != 0xFFFFFFFFu;
        load_k<D, FP8>(kbase + static_cast<size_t>(next_have ? next_row : 0u) * (D * L::esz), g, j, kr);
      }
      // softmax of the tile: lane (g, j) has heads g (and g + 8), tokens 8 r + 2 j and + 1
      uint32_t hi[HT][2], lo[HT][2];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float z[4];
        float top = m[h];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 8 * (i >> 1) + 2 * j + (i & 1);
          z[i] = s[i >> 1][2 * h + (i & 1)] * qs[h];
          if (tok >= live) z[i] = __int_as_float(0xff800000);
          top = fmaxf(top, z[i]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (__any_sync(0xffffffffu, top > m[h])) {
          const float keep = m[h] == top ? 1.f : exp2f(m[h] - top);   // top > -inf here, or m == top
          l[h] *= keep;
          const float k0 = __shfl_sync(0xffffffffu, keep, 8 * j), k1 = __shfl_sync(0xffffffffu, keep, 8 * j + 4);
#pragma unroll
          for (int i = 0; i < L::mt; ++i) {
            o[h][i][0] *= k0;
            o[h][i][1] *= k1;
            o[h][i][2] *= k0;
            o[h][i][3] *= k1;
          }
          m[h] = top;
        }
        const float base = m[h] == __int_as_float(0xff800000) ? 0.f : m[h];
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = exp2f(z[i] - base);
          l[h] += p[i];
          p[i] *= kPScale;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (FP8) {
            hi[h][r] = pack_f16x2(p[2 * r], p[2 * r + 1]);
            const __half2 t2 = *reinterpret_cast<const __half2*>(&hi[h][r]);
            lo[h][r] = pack_f16x2(p[2 * r] - __low2float(t2), p[2 * r + 1] - __high2float(t2));
          } else {
            hi[h][r] = pack_bf16x2(p[2 * r], p[2 * r + 1]);
            lo[h][r] = pack_bf16x2(p[2 * r] - __uint_as_float(hi[h][r] << 16),
                                   p[2 * r + 1] - __uint_as_float(hi[h][r] & 0xFFFF0000u));
          }
        }
      }
      if (live < 16) {   // what lies behind the sequence's end may be anything, and 0 x NaN is NaN
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (2 * j + (r & 1) + 8 * (r >> 1) >= live) {
#pragma unroll
            for (int w = 0; w < L::vwords; ++w) vr[r][w] = 0u;
          }
      }
#pragma unroll
      for (int w = 0; w < L::vwords; ++w) {
        if (FP8) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {   // columns 4 w + 2 half, + 1 of the lane's share
            const uint32_t x = __byte_perm(vr[0][w], vr[1][w], half ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(vr[2][w], vr[3][w], half ? 0x7362 : 0x5140);
            const uint32_t va[4] = {e4m3x2_to_f16x2(static_cast<uint16_t>(x & 0xFFFFu)),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(x >> 16)),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(y & 0xFFFFu)),
                                    e4m3x2_to_f16x2(static_cast<uint16_t>(y >> 16))};
#pragma unroll
            for (int h = 0; h < HT; ++h) {
              mma_f16(o[h][2 * w + half], va, hi[h][0], hi[h][1]);
              mma_f16(o[h][2 * w + half], va, lo[h][0], lo[h][1]);
            }
          }
        } else {
          uint32_t va[4] = {__byte_perm(vr[0][w], vr[1][w], 0x5410), __byte_perm(vr[0][w], vr[1][w], 0x7632),
                                  __byte_perm(vr[2][w], vr[3][w], 0x5410), __byte_perm(vr[2][w], vr[3][w], 0x7632)};
#pragma unroll
          for (int h = 0; h < HT; ++h) mma_bf16(o[h][w], va, hi[h][0], hi[h][1]);
          if (careful) {
#pragma unroll
            for (int i = 0; i < 4; ++i) va[i] = finite_bf16x2(va[i]);
          }
#pragma unroll
          for (int h = 0; h < HT; ++h) mma_bf16(o[h][w], va, lo[h][0], lo[h][1]);
        }
      }
      if (t + 1 < t_end)
        load_v<D, FP8>(vbase + static_cast<size_t>(next_have ? next_row : 0u) * (D * L::esz), g, j, vr);
      have = next_have;
    }
    if (!FP8 && !careful) {
      bool nan = false;
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int i = 0; i < L::mt; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) nan |= o[h][i][e] != o[h][i][e];
      if (__any_sync(0xffffffffu, nan)) {
        careful = true;
        goto again;
      }
    }
    // lane (g, j): o[h][..] has heads 8 h + 2 j (elements 0, 2) and + 1 (1, 3), columns v_col and + 1
    const bool whole = tile == 0 && t_end == nt;
    const int slot = x == x0 ? 0 : 1;
    float* part = a.parts + (static_cast<size_t>(gw) * 2 + slot) * part_floats<D, HT>();
    const float vs = FP8 ? __ldg(a.v_scale + hk) / kPScale : 1.f;
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      const int head = row0 + 8 * h + g;   // of the group
      if (j == 0) {
        if (!whole) {
          part[8 * h + g] = m[h];
          part[H + 8 * h + g] = l[h];
        } else if (a.lse && head < a.G) {
          a.lse[static_cast<size_t>(b) * a.Hq + static_cast<size_t>(hk) * a.G + head] = (m[h] + log2f(l[h])) * kLn2;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float le = __shfl_sync(0xffffffffu, l[h], 8 * j + 4 * e);
        const int hd = row0 + 8 * h + 2 * j + e;
        if (whole && hd >= a.G) continue;
        const size_t at = (static_cast<size_t>(b) * a.Hq + static_cast<size_t>(hk) * a.G + hd) * D;
        const float f = !whole ? vs : (le == 0.f ? 0.f : vs * gate_of(a, b, hk * a.G + hd) / le);
#pragma unroll
        for (int i = 0; i < L::mt; ++i) {
          const int col = FP8 ? v_col<D, FP8>(g, i >> 1) + 2 * (i & 1) : v_col<D, FP8>(g, i);
          if (whole) store2(static_cast<TO*>(a.out) + at + col, o[h][i][e] * f, o[h][i][2 + e] * f);
          else store2(part + 2 * H + (8 * h + 2 * j + e) * D + col, o[h][i][e] * f, o[h][i][2 + e] * f);
        }
      }
    }
    // on to the next group or sequence
    x += t_end - tile;
    if (x < x1) {
      tile = 0;
      if (++u == units) {
        u = 0;
        do {
          n = seq_len(a, ++b);
          nt = tiles_of(n);
        } while (nt == 0);
      }
    }
  }
}

// Joins the parts of the groups that were cut, one block per (sequence, query head), and writes the rows of empty
// sequences.
template <int D, int HT, typename TO>
__global__ void __launch_bounds__(kThreads) join_kernel(AttnArgs a) {
  constexpr int H = 8 * HT, kCols = D / 32;
  __shared__ long long scan[kWarps];
  __shared__ long long start_of_b;
  __shared__ float red[kWarps][D + 2];
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x - b * a.Hq;
  const int hk = hq / a.G, in_group = hq - hk * a.G, gt = in_group / H, head = in_group - gt * H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = a.Hkv * a.gtiles;
  const int per = (a.B + kThreads - 1) / kThreads, b_lo = threadIdx.x * per;
  const int b_hi = b_lo + per < a.B ? b_lo + per : a.B;
  long long mine = 0;
  for (int i = b_lo; i < b_hi; ++i) mine += static_cast<long long>(tiles_of(seq_len(a, i))) * units;
  long long total;
  const long long pre = block_prefix(mine, scan, total);
  if (b >= b_lo && b < b_hi) {
    long long p = pre;
    for (int i = b_lo; i < b; ++i) p += static_cast<long long>(tiles_of(seq_len(a, i))) * units;
    start_of_b = p;
  }
  __syncthreads();
  const int nt = tiles_of(seq_len(a, b));
  TO* out = static_cast<TO*>(a.out) + (static_cast<size_t>(b) * a.Hq + hq) * D;
  // every thread of the first kernel's grid is done, and its writes are visible, behind this line
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (nt == 0) {
    for (int c = threadIdx.x * 2; c < D; c += kThreads * 2) store2(out + c, 0.f, 0.f);
    if (a.lse && threadIdx.x == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = __int_as_float(0xff800000);
    return;
  }
  const long long p0 = start_of_b + static_cast<long long>(hk * a.gtiles + gt) * nt, p1 = p0 + nt;
  const Pieces pieces(total, a.warps);
  const int w0 = pieces.owner(p0), w1 = pieces.owner(p1 - 1);
  if (w0 == w1) return;   // written whole
  const int first_slot = pieces.start(w0) == p0 ? 0 : 1;
  auto part_of = [&](int w) -> const float* {
    return a.parts + (static_cast<size_t>(w) * 2 + (w == w0 ? first_slot : 0)) * part_floats<D, HT>();
  };
  float m = __int_as_float(0xff800000);
  for (int w = w0 + static_cast<int>(threadIdx.x); w <= w1; w += kThreads) m = fmaxf(m, __ldcg(part_of(w) + head));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp][0] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red[w][0]);
  __syncthreads();
  const float base = m == __int_as_float(0xff800000) ? 0.f : m;
  float l = 0.f, acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
#pragma unroll 8
  for (int w = w0 + warp; w <= w1; w += kWarps) {
    const float* p = part_of(w);
    const float k = exp2f(__ldcg(p + head) - base);
    l = fmaf(__ldcg(p + H + head), k, l);
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = fmaf(__ldcg(p + 2 * H + head * D + c * 32 + lane), k, acc[c]);
  }
  if (lane == 0) red[warp][D] = l;
#pragma unroll
  for (int c = 0; c < kCols; ++c) red[warp][c * 32 + lane] = acc[c];
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) l += red[w][D];
  const float f = l == 0.f ? 0.f : gate_of(a, b, hq) / l;
  for (int c = threadIdx.x * 2; c < D; c += kThreads * 2) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      x += red[w][c];
      y += red[w][c + 1];
    }
    store2(out + c, x * f, y * f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = (m + log2f(l)) * kLn2;
}

template <int D, bool FP8, int HT, typename TO>
zmoe_status launch(AttnArgs a, cudaStream_t s) {
  const int blocks = num_sms() * (HT == 1 ? 3 : 2);
  a.warps = blocks * kWarps;
  static_assert((HT == 1 ? 3 : 2) * kWarps <= kMaxWarpsPerSm, "the workspace holds the warps' parts");
  attn_kernel<D, FP8, HT, TO><<<blocks, kThreads, 0, s>>>(a);
  zmoe_status st = check_launch("zmoe_paged_attention");
  if (st != ZMOE_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.Hq);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, join_kernel<D, HT, TO>, a);
  return check_launch("zmoe_paged_attention (join)");
}

template <int D, bool FP8>
zmoe_status launch_out(AttnArgs& a, bool bf16_out, cudaStream_t s) {
  if (a.G <= 8) {
    a.gtiles = 1;
    return bf16_out ? launch<D, FP8, 1, uint16_t>(a, s) : launch<D, FP8, 1, float>(a, s);
  }
  a.gtiles = (a.G + 15) / 16;
  return bf16_out ? launch<D, FP8, 2, uint16_t>(a, s) : launch<D, FP8, 2, float>(a, s);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace zmoe

extern "C" {

size_t zmoe_paged_attention_workspace_size(int B, int Hq, int Hkv, int D) {
  using namespace zmoe;
  if (B <= 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  const int H = Hq / Hkv <= 8 ? 8 : 16;
  return static_cast<size_t>(num_sms()) * kMaxWarpsPerSm * 2 * H * (D + 2) * 4;
}

zmoe_status zmoe_paged_attention(const void* q, const void* k_cache, const void* v_cache, zmoe_dtype kv_dtype,
                                 const float* k_scale, const float* v_scale, const int32_t* page_table,
                                 const int32_t* lens, const float* gate, float scale, int B, int Hq, int Hkv, int D,
                                 int max_pages, int n_pages, int page_size, void* out, zmoe_dtype out_dtype, float* lse,
                                 void* workspace, size_t ws_bytes, zmoe_stream_t stream) {
  ZMOE_TRACE("zmoe_paged_attention");
  using namespace zmoe;
  ZMOE_REQUIRE(kv_dtype == ZMOE_BF16 || kv_dtype == ZMOE_E4M3, "zmoe_paged_attention: the cache is bf16 or E4M3");
  ZMOE_REQUIRE(dtype_ok(out_dtype), "zmoe_paged_attention: the output is f32 or bf16");
  ZMOE_REQUIRE(B >= 0 && Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0, "zmoe_paged_attention: Hq must be a multiple of Hkv");
  ZMOE_REQUIRE(D >= 1, "zmoe_paged_attention: bad D");
  ZMOE_REQUIRE(page_size >= 16 && page_size % 16 == 0, "zmoe_paged_attention: page_size must be a multiple of 16");
  ZMOE_REQUIRE(max_pages >= 0 && n_pages >= 1, "zmoe_paged_attention: bad max_pages or n_pages");
  ZMOE_REQUIRE(scale == scale, "zmoe_paged_attention: scale is NaN");
  if (B == 0) return ZMOE_OK;
  ZMOE_REQUIRE(q && k_cache && v_cache && lens && out && (page_table || max_pages == 0),
               "zmoe_paged_attention: NULL pointer");
  ZMOE_REQUIRE(kv_dtype == ZMOE_BF16 || (k_scale && v_scale),
               "zmoe_paged_attention: an E4M3 cache needs k_scale and v_scale");
  if (D != 64 && D != 128) return fail(ZMOE_ERR_UNSUPPORTED, "zmoe_paged_attention: D must be 64 or 128");
  ZMOE_REQUIRE(aligned16(q) && aligned16(k_cache) && aligned16(v_cache) && aligned16(out) && aligned4(k_scale) &&
                   aligned4(v_scale) && aligned4(page_table) && aligned4(lens) && aligned4(gate) && aligned4(lse),
               "zmoe_paged_attention: q, the caches and out must be 16-byte aligned");
  ZMOE_REQUIRE(static_cast<long long>(max_pages) * page_size <= 0x7fffffffLL,
               "zmoe_paged_attention: max_pages * page_size overflows int32");
  ZMOE_REQUIRE(static_cast<unsigned long long>(n_pages) * Hkv * page_size < 0xffffffffULL,
               "zmoe_paged_attention: n_pages * Hkv * page_size overflows 32 bits");
  ZMOE_REQUIRE(static_cast<long long>(B) * Hq <= 0x7fffffffLL, "zmoe_paged_attention: B * Hq overflows int32");
  if (!workspace || ws_bytes < zmoe_paged_attention_workspace_size(B, Hq, Hkv, D))
    return fail(ZMOE_ERR_WORKSPACE_TOO_SMALL,
                "zmoe_paged_attention: workspace smaller than zmoe_paged_attention_workspace_size()");
  ZMOE_REQUIRE(aligned16(workspace), "zmoe_paged_attention: workspace must be 16-byte aligned");
  clear_error();
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = k_cache; a.v = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
  a.table = page_table; a.lens = lens; a.gate = gate; a.scale = scale;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
  a.max_pages = max_pages; a.n_pages = n_pages; a.page_size = page_size;
  a.out = out; a.lse = lse; a.parts = static_cast<float*>(workspace);
  a.errors = device_error_counter();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = out_dtype == ZMOE_BF16;
  if (kv_dtype == ZMOE_E4M3) return D == 64 ? launch_out<64, true>(a, bf, s) : launch_out<128, true>(a, bf, s);
  return D == 64 ? launch_out<64, false>(a, bf, s) : launch_out<128, false>(a, bf, s);
}

}  // extern "C"
