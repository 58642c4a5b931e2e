// zmoe_paged_attention: attention of one new token per sequence over a paged key-value cache.
//
// ZONOS2 Technical Report digest, "method overview and architecture", item 5 (grouped-query attention with
// headwise gating).  Per sequence b with n = lens[b] cached tokens and query head i of key-value head g:
//   s_t = scale q_i . k_t;   o_i = sum_t exp(s_t) v_t / sum_t exp(s_t),  t < n;   lse_i = log sum_t exp(s_t)
//   out_i = sigmoid(gate_i) o_i                                               (o = 0, lse = -inf when n = 0)
//
// Bound by HBM: every cached key and value is read once (per 8 or 16 query heads of a group).  A warp takes 8 KB of
// them at a time, a step of 16 (bf16, 128 columns) to 64 tokens; each 16 of these lie in one page, and their keys
// and their values come by one TMA copy each into the warp's own ring in shared memory (128-byte swizzle, an mbarrier
// a step, two steps), so 12 warps keep up to 192 KB an SM in flight, and no warp waits for another.
//   scores  S = Q K^T:      m16n8k16, 16 rows of query heads (8 or 16 in use), 8 tokens, 16 columns;
//   output  O^T = V^T P^T:  m16n8k16, 16 columns of V, 8 query heads, 16 tokens.
// (A tcgen05 product has at least 64 rows, of which a group of 4 or 8 heads would fill as many, and its accumulator lies
// in tensor memory, from where the softmax would have to fetch it; the warp's product leaves S in registers.  Groups of more
// than 16 heads read the cache once for each 16 of them: 64 heads a group would fill such a product, which is not built.)
// The contraction index of a tensor-core product may be permuted as long as both operands agree, so each lane's
// share of a key row is 16-byte chunks, each lane's share of the output is 8 contiguous columns, and the swizzle
// keeps both free of bank conflicts.  S leaves the first product in the layout that the second takes P^T in.  The
// maximum and the sum of the softmax run along in registers.
//
// Work is split over the cache's length: the (sequence, group, 16-token tile) triples are one line of tiles, cut into
// equal pieces, one a warp, so that ragged lengths balance; the ring runs ahead over the ends of sequences.  A warp
// writes the groups that lie within its piece; of a group that is cut it leaves a part (maximum, sum, O).  Where groups
// are cut into many, a CTA's warps take neighbouring pieces and join their parts first.  A second kernel, launched to
// start early (programmatic dependent launch), joins what is left in a fixed order.
//
// Measured: 64 sequences of 1 to 4096 tokens (134k), 16 + 4 heads of 128, bf16: 55 us, 5.0 TB/s; 4 sequences, 286k
// tokens, 32 + 4 heads of 128, E4M3: 61 us, 4.8 TB/s; one sequence of 431 tokens: 8.5 us; one of 20000 with 8 + 1 heads:
// 14.3 us.  A longer cache adds at 6.1 (bf16) and 7 TB/s (E4M3); about 12 us are the two launches, the lengths' prefix,
// the first copies and the join.
//
// P is split into 16-bit terms, P = P_1 + P_2 (+ P_3), and the second product runs for each: one bf16 term alone would
// cost 2^-9 of every weight.  Two bf16 terms leave 2^-16 of it, which a bf16 output does not show; an f32 output takes
// a third, and an f16 pair (8-bit cache) has 22 bits.  The bf16 terms are cut, not rounded, so that none is negative,
// and are at least 2^-126 where P is not 0: an infinite value then meets positive weights only and stays an infinity,
// as in the formula.  An 8-bit cache is expanded to f16, exactly; its queries are scaled by a power of two per head to
// use f16's range, and so is P.
#include "sm100_ptx.cuh"
#include "vectors.cuh"

namespace zmoe {

unsigned int* device_timeout_counter();

namespace {

using namespace ptx;

constexpr int kJoinThreads = 256;
constexpr int kMaxWarps = 12;        // of a CTA of the first kernel
constexpr uint64_t kWaitNs = 2000000000ull;   // a wait for a copy gives up after this
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
  float* parts;           // [warps][2] of {m[H], l[H], O[H][D]}, H = 8 HT: what the first kernel leaves to the second;
                          // or, where its CTAs join their warps' parts, [ctas][2], and behind them [warps] of the parts
                          // that a warp is done with before its last one
  int ctas;               // of the first kernel
  int together;           // log2 of the query heads of a group that a block of the second kernel joins
  unsigned int *errors, *timeouts;
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

// Four E4M3 values -> two f16 pairs; exact.
__device__ __forceinline__ void widen_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 2^x, 0 below 2^-126.
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The length of sequence b; one beyond the table's pages is an error and cut to them.  EARLY: read past the L1 cache,
// by a kernel that has not waited for the one before it yet.
template <bool EARLY = false>
__device__ __forceinline__ int seq_len(const AttnArgs& a, int b) {
  const int n = EARLY ? __ldcg(a.lens + b) : a.lens[b];
  const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
  return n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
}

__device__ __forceinline__ int tiles_of(int n) { return static_cast<int>((static_cast<unsigned>(n) + 15u) >> 4); }

__device__ __forceinline__ long long divide(long long x, long long y) {   // of numbers that are not negative
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// `total` tiles in `count` pieces, none empty: the first `more` pieces have one tile more.
struct Pieces {
  int count;
  long long size, more;

  __device__ __forceinline__ Pieces(long long total, int most)
      : count(total < most ? static_cast<int>(total) : most), size(divide(total, count)), more(total - size * count) {}
  __device__ __forceinline__ long long start(long long w) const { return w * size + (w < more ? w : more); }
  __device__ __forceinline__ int owner(long long x) const {   // the piece that tile x is in
    const long long big = more * (size + 1);
    return static_cast<int>(x < big ? divide(x, size + 1) : more + divide(x - big, size));
  }
};

// Exclusive prefix over the block's threads of `mine`; every thread receives the total.
template <int WARPS>
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
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  return before + inc - mine;
}

// A part of a group (sequence b, group u) as a warp leaves it; null: none.
struct Segment {
  const float* part;
  int b, u;
  bool begins, ends;   // with the group's first tile, with its last
};

// Warps of a CTA of the first kernel, one CTA an SM: 168 or 255 registers a thread.
template <int HT>
__host__ __device__ constexpr int warps_of() {
  return HT == 1 ? 12 : 8;
}

template <int D, int HT>
__host__ __device__ constexpr int part_floats() {
  return 8 * HT * (D + 2);
}

// How tiles of an 8-bit or a bf16 cache are read.  A tile's rows lie in shared memory one after another as lines of
// 128 bytes, each line's 16-byte chunks exchanged by the line's number (modulo 8).
template <int D, bool FP8, int HT>
struct Lay {
  static constexpr int esz = FP8 ? 1 : 2;
  static constexpr int row = D * esz;              // bytes
  static constexpr int kvecs = row / 64;           // 16-byte vectors of a key row per lane (4 lanes a row)
  static constexpr int vwords = row / 32;          // 32-bit words of a value row per lane (8 lanes a row)
  static constexpr int steps = D / 16;             // 16-column steps of the first product
  static constexpr int mt = D / 16;                // 16-column tiles of the output
  static constexpr int half = 16 * row;            // bytes of a tile's keys or values
  static constexpr int tiles = 4096 / half;        // tiles of a step
  static constexpr int slot = 8192;                // bytes of a step: its keys, its values
  static constexpr int warps = warps_of<HT>();
  static constexpr int slots = HT == 1 ? 2 : 3;
  static constexpr int smem = warps * slots * slot + 1024;   // the rings start on 1024 bytes
  static_assert(half % 1024 == 0 && tiles >= 1, "whole swizzle atoms");
  static_assert(part_floats<D, HT>() * 4 <= slots * slot && warps <= kMaxWarps, "a part fits the warp's ring");

  // Chunk c of lane j's share of a key row, in 16-byte chunks of the row: eight neighbouring lanes, which have two
  // rows, reach all banks.
  __device__ __forceinline__ static int k_chunk(int c, int j) {
    if (row == 256) return (c >> 1) * 8 + (j >> 1) * 4 + (c & 1) * 2 + (j & 1);
    return row == 128 ? 2 * j + c : j;
  }
  // Byte `at` of token r's row within a tile.
  __device__ __forceinline__ static uint32_t place(int r, int at) {
    const uint32_t x = static_cast<uint32_t>(r * row + at);
    return x ^ (((x >> 7) & 7u) << 4);
  }
};

// A tile's rows from line `at` of the cache on.
__device__ __forceinline__ void tma_lines(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int at) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(at)
      : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(p));
  return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(p));
  return r;
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
  return a.gate ? 1.f / (1.f + expf(-a.gate[static_cast<size_t>(b) * a.Hq + head])) : 1.f;
}

// Do the CTAs of the first kernel join the parts of their warps?  It costs every CTA 2 to 3 us at its end, and saves the
// second kernel a factor of 12 (or 8) where a group is cut into many parts: 27 parts a group took 8.3 us a call without
// and 9.6 with, 7 parts 54.6 and 57.2, 111 parts 65.5 and 61.6, 1250 parts 71 and 14.3.
__device__ __forceinline__ bool joined_early(const AttnArgs& a, const Pieces& pieces) {
  return pieces.count > 64LL * a.B * a.Hkv * a.gtiles;
}

template <int D, bool FP8, int HT, typename TO>
__global__ void __launch_bounds__(32 * Lay<D, FP8, HT>::warps, 1)
    attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs a) {
  using L = Lay<D, FP8, HT>;
  constexpr int H = 8 * HT, kWarps = L::warps, kThreads = 32 * kWarps;
  constexpr int kTerms = !FP8 && sizeof(TO) == 4 ? 3 : 2;
  constexpr float kPScale = FP8 ? 32768.f : 1.f;   // f16 holds P in [0, 2^15]: weights down to 2^-39 survive
  extern __shared__ unsigned char ring_raw[];
  __shared__ uint64_t bars[kWarps][L::slots];
  __shared__ long long scan[kWarps];
  __shared__ int at_b[kWarps];
  __shared__ long long at_off[kWarps];
  __shared__ Segment segments[2 * kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  const int units = a.Hkv * a.gtiles;
  uint64_t* bar = bars[warp];
  unsigned char* const rings = ring_raw + ((1024u - (smem_u32(ring_raw) & 1023u)) & 1023u);
  const uint32_t ring = smem_u32(rings) + static_cast<uint32_t>(warp * L::slots * L::slot);
  if (lane < 2) segments[2 * warp + lane].part = nullptr;
  if (lane == 0) {
    asm volatile("prefetch.tensormap [%0];\n\tprefetch.tensormap [%1];" ::"l"(reinterpret_cast<uint64_t>(&kmap)),
                 "l"(reinterpret_cast<uint64_t>(&vmap)));
    for (int i = 0; i < L::slots; ++i) mbar_init(bar + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
  }
  // what came before is complete, and only now may the second kernel begin: it reads the lengths before its own wait
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  // the line of tiles: sequence by sequence, in each the groups, in each the tiles
  const int per = (a.B + kThreads - 1) / kThreads, b_lo = threadIdx.x * per;
  const int b_hi = b_lo + per < a.B ? b_lo + per : a.B;
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    mine += static_cast<long long>(tiles_of(seq_len(a, b))) * units;
    if (blockIdx.x == 0 && a.lens[b] > static_cast<long long>(a.max_pages) * a.page_size)
      record_device_error(a.errors);
  }
  long long total;
  const long long pre = block_prefix<kWarps>(mine, scan, total);
  if (total == 0) return;
  const Pieces pieces(total, a.ctas * kWarps);
  // neighbouring pieces go to a CTA that joins them, or to neighbouring SMs
  const bool early = joined_early(a, pieces);
  const int first_piece = early ? blockIdx.x * kWarps : blockIdx.x, next_piece = early ? 1 : a.ctas;
  if (first_piece >= pieces.count) return;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int i = first_piece + w * next_piece;
    const long long x = pieces.start(i);
    if (i < pieces.count && x >= pre && x < pre + mine) {
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
  const int gw = first_piece + warp * next_piece;
  const bool busy = gw < pieces.count;
  const int piece = busy ? static_cast<int>(pieces.start(gw + 1) - pieces.start(gw)) : 0;   // tiles (2^31 would take hours)
  int b = busy ? at_b[warp] : 0, n = seq_len(a, b), nt = tiles_of(n);
  int u = busy ? static_cast<int>(divide(at_off[warp], nt)) : 0;
  int tile = busy ? static_cast<int>(at_off[warp] - static_cast<long long>(u) * nt) : 0;

  // The feeder runs ahead of the products: the keys and values of a step's tiles into the next slot.
  const int tpp = a.page_size >> 4;   // tiles per page
  int f_b = b, f_u = u, f_tile = tile, f_nt = nt, f_win = tile, f_slot = 0;
  int f_left = piece;                 // tiles to feed
  uint32_t f_have = 0;                // which tiles of the steps in the ring have a page: the oldest step lowest
  // cache lines of the 32 tiles from f_win on (lane i: tile f_win + i); -1: no page
  auto lines_from = [&](int win) -> int {
    const int t = win + lane;
    int line = -1;
    if (t < f_nt && t - f_tile < f_left) {
      const int col = t / tpp;
      const int pid = a.table[static_cast<size_t>(f_b) * a.max_pages + col];
      if (pid >= 0 && pid < a.n_pages)
        line = ((pid * a.Hkv + f_u / a.gtiles) * a.page_size + (t - col * tpp) * 16) >> (L::row == 64 ? 1 : 0);
      else if (f_u == 0 && (t == f_tile || t == col * tpp))
        record_device_error(a.errors);
    }
    return line;
  };
  int f_lines = lines_from(f_win);
  auto feed = [&](int ahead) {   // ahead: steps in the ring before this one
    if (f_left == 0) return;
    const int rest = f_nt - f_tile < f_left ? f_nt - f_tile : f_left, here = rest < L::tiles ? rest : L::tiles;
    uint64_t* full = bar + f_slot;
    const uint32_t dst = ring + f_slot * L::slot;
    if (lane == 0) mbar_expect_tx(full, here * 2 * L::half);
    uint32_t have = 0;
#pragma unroll
    for (int i = 0; i < L::tiles; ++i) {
      const int line = __shfl_sync(0xffffffffu, f_lines, f_tile - f_win + i);
      if (line >= 0) have |= 1u << i;
      if (lane == 0 && i < here) {
        const int at = line >= 0 ? line : 0;   // any rows in place of none: these tokens do not count
        tma_lines(dst + i * L::half, &kmap, full, at);
        tma_lines(dst + 4096 + i * L::half, &vmap, full, at);
      }
    }
    f_have |= have << (ahead * L::tiles);
    if (++f_slot == L::slots) f_slot = 0;
    f_left -= here;
    f_tile += here;
    if (f_tile == f_nt && f_left > 0) {   // on to the next group or sequence
      f_tile = 0;
      if (++f_u == units) {
        f_u = 0;
        do {
          f_nt = tiles_of(seq_len(a, ++f_b));
        } while (f_nt == 0);
      }
      f_lines = lines_from(f_win = 0);
    } else if (f_tile - f_win == 32) {
      f_lines = lines_from(f_win = f_tile);
    }
  };
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < L::slots; ++i) feed(i);
  int slot = 0;
  uint32_t parity = 0;
  // The next slot's copy has landed (false: it did not come in time).
  volatile int never = 0;
  auto landed = [&]() {
    const bool ok = mbar_wait(bar + slot, parity, &never, kWaitNs);
    return __all_sync(0xffffffffu, ok);
  };
  bool gave_up = false;
  for (int todo = piece; todo > 0;) {
    const int t_end = todo < nt - tile ? tile + todo : nt;
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
        // the columns of lane j's key chunks: 8 a chunk (bf16), 16 (8-bit cache)
        const int col = FP8 ? L::k_chunk(c >> 1, j) * 16 + (c & 1) * 8 : L::k_chunk(c, j) * 8;
        raw[c] = on ? *reinterpret_cast<const uint4*>(qr + col) : make_uint4(0u, 0u, 0u, 0u);
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
        // the largest magnitude goes to [2^14, 2^15), unless it is below 2^-86: such a query scores 0 anyway
        const int bits = static_cast<int>(__float_as_uint(top) >> 23), ex = bits == 255 ? 0 : (bits < 41 ? 100 : 141 - bits);
        const float up = __int_as_float((127 + ex) << 23);
        if (r < HT) qs[r] = a.scale * kLog2e * a.k_scale[hk] * __int_as_float((127 - ex) << 23);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float f[8];
          unpack_bf16x8(raw[c], f);
          raw[c] = make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up),
                              pack_f16x2(f[4] * up, f[5] * up), pack_f16x2(f[6] * up, f[7] * up));
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
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      m[h] = __int_as_float(0xff800000);
      l[h] = 0.f;
#pragma unroll
      for (int i = 0; i < L::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][i][e] = 0.f;
    }
#pragma unroll 1
    for (int t = tile; t < t_end; t += L::tiles) {
      if (!landed()) {
        gave_up = true;
        break;
      }
      const uint32_t base = ring + slot * L::slot;
      // tokens of each tile that count
      int live[L::tiles];
      bool full = true;
#pragma unroll
      for (int i = 0; i < L::tiles; ++i) {
        const int left = t + i < t_end && ((f_have >> i) & 1u) ? n - (t + i) * 16 : 0;
        live[i] = left < 16 ? left : 16;
        full = full && left >= 16;
      }
      float s[L::tiles][2][4];
#pragma unroll
      for (int i = 0; i < L::tiles; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][r][e] = 0.f;
      // neighbouring products go to different sums
#pragma unroll
      for (int c = 0; c < L::kvecs; ++c) {
        uint4 kr[L::tiles][2];
#pragma unroll
        for (int i = 0; i < L::tiles; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            kr[i][r] = lds128(base + i * L::half + L::place(g + 8 * r, L::k_chunk(c, j) * 16));
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < L::tiles; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4& v = kr[i][r];
              if (FP8) {
                uint32_t b0, b1;
                widen_e4m3x4(q == 0 ? v.x : (q == 1 ? v.y : (q == 2 ? v.z : v.w)), b0, b1);
                mma_f16(s[i][r], qf[4 * c + q], b0, b1);
              } else if (q < 2) {
                mma_bf16(s[i][r], qf[2 * c + q], q ? v.z : v.x, q ? v.w : v.y);
              }
            }
      }
      // softmax of the step: lane (g, j) has heads g (and g + 8), of each tile the tokens 8 r + 2 j and + 1
      uint32_t pt[L::tiles][HT][kTerms][2];   // P's terms
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float z[L::tiles][4];
        float top = m[h];
#pragma unroll
        for (int i = 0; i < L::tiles; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[i][e] = s[i][e >> 1][2 * h + (e & 1)] * qs[h];
            if (!full && 8 * (e >> 1) + 2 * j + (e & 1) >= live[i]) z[i][e] = __int_as_float(0xff800000);
            top = fmaxf(top, z[i][e]);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (__any_sync(0xffffffffu, top > m[h])) {
          const float keep = m[h] == top ? 1.f : pow2(m[h] - top);   // top > -inf here, or m == top
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
        const float zero = m[h] == __int_as_float(0xff800000) ? 0.f : m[h];
#pragma unroll
        for (int i = 0; i < L::tiles; ++i) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = pow2(z[i][e] - zero);
            l[h] += p[e];
            p[e] *= kPScale;
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = p[2 * r], p1 = p[2 * r + 1];
            if (FP8) {
              const uint32_t w = pack_f16x2(p0, p1);
              const __half2 t2 = *reinterpret_cast<const __half2*>(&w);
              pt[i][h][0][r] = w;
              pt[i][h][1][r] = pack_f16x2(p0 - __low2float(t2), p1 - __high2float(t2));
            } else {
              const float least0 = fminf(p0, 1.17549435e-38f), least1 = fminf(p1, 1.17549435e-38f);   // 2^-126
              float r0 = p0, r1 = p1;   // what is left of P
#pragma unroll
              for (int t = 0; t < kTerms; ++t) {
                if (t == kTerms - 1) {
                  pt[i][h][t][r] = round_bf16x2(r0, r1);
                } else {
                  const uint32_t x = __float_as_uint(r0), y = __float_as_uint(r1);
                  pt[i][h][t][r] = __byte_perm(x, y, 0x7632);
                  r0 = fmaxf(r0 - __uint_as_float(x & 0xFFFF0000u), least0);
                  r1 = fmaxf(r1 - __uint_as_float(y & 0xFFFF0000u), least1);
                }
              }
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < L::tiles; ++i) {
        uint32_t vr[4][L::vwords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = 2 * j + (r & 1) + 8 * (r >> 1);
          const uint32_t from = base + 4096 + i * L::half;
          if (L::vwords == 2) {
            const uint2 w = lds64(from + L::place(tok, g * 8));
            vr[r][0] = w.x;
            vr[r][1] = w.y;
          } else {
#pragma unroll
            for (int c = 0; c < L::vwords / 4; ++c) {
              const uint4 w = lds128(from + L::place(tok, c * 128 + g * 16));
              vr[r][4 * c] = w.x;
              vr[r][4 * c + 1] = w.y;
              vr[r][4 * c + 2] = w.z;
              vr[r][4 * c + 3] = w.w;
            }
          }
        }
        if (live[i] < 16) {   // what lies behind the sequence's end may be anything, and 0 x NaN is NaN
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (2 * j + (r & 1) + 8 * (r >> 1) >= live[i]) {
#pragma unroll
              for (int w = 0; w < L::vwords; ++w) vr[r][w] = 0u;
            }
        }
        // the column tiles of kSide words side by side: a tile's products are apart from one another
        constexpr int kSide = FP8 ? 2 : 4, kTiles = FP8 ? 2 * kSide : kSide;
#pragma unroll
        for (int w0 = 0; w0 < L::vwords; w0 += kSide) {
          uint32_t va[kTiles][4];
#pragma unroll
          for (int k = 0; k < kSide; ++k) {
            const int w = w0 + k;
            if (FP8) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {   // columns 4 w + 2 half, + 1 of the lane's share
                uint32_t(&t)[4] = va[(2 * k + half) % kTiles];
                widen_e4m3x4(__byte_perm(vr[0][w], vr[1][w], half ? 0x7362 : 0x5140), t[0], t[1]);
                widen_e4m3x4(__byte_perm(vr[2][w], vr[3][w], half ? 0x7362 : 0x5140), t[2], t[3]);
              }
            } else {
              uint32_t(&t)[4] = va[k % kTiles];
              t[0] = __byte_perm(vr[0][w], vr[1][w], 0x5410);
              t[1] = __byte_perm(vr[0][w], vr[1][w], 0x7632);
              t[2] = __byte_perm(vr[2][w], vr[3][w], 0x5410);
              t[3] = __byte_perm(vr[2][w], vr[3][w], 0x7632);
            }
          }
          const int o0 = FP8 ? 2 * w0 : w0;
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
#pragma unroll
            for (int h = 0; h < HT; ++h)
#pragma unroll
              for (int k = 0; k < kTiles; ++k) {
                if (FP8) mma_f16(o[h][o0 + k], va[k], pt[i][h][t][0], pt[i][h][t][1]);
                else mma_bf16(o[h][o0 + k], va[k], pt[i][h][t][0], pt[i][h][t][1]);
              }
        }
      }
      // every lane has read the slot: it is filled again
      __syncwarp();
      f_have >>= L::tiles;
      feed(L::slots - 1);
      if (++slot == L::slots) {
        slot = 0;
        parity ^= 1;
      }
    }
    if (gave_up) break;
    // lane (g, j): o[h][..] has heads 8 h + 2 j (elements 0, 2) and + 1 (1, 3), columns v_col and + 1
    const bool whole = tile == 0 && t_end == nt;
    const int part_slot = todo == piece ? 0 : 1;
    const bool last = todo == t_end - tile;
    float* part;
    if (early) {   // the last part lies in the ring, which is free then, one before it in memory
      part = last ? reinterpret_cast<float*>(rings + warp * L::slots * L::slot)
                  : a.parts + (static_cast<size_t>(a.ctas) * 2 + gw) * part_floats<D, HT>();
      if (!whole && lane == 0) segments[2 * warp + part_slot] = Segment{part, b, u, tile == 0, t_end == nt};
    } else {
      part = a.parts + (static_cast<size_t>(gw) * 2 + part_slot) * part_floats<D, HT>();
    }
    const float vs = FP8 ? a.v_scale[hk] / kPScale : 1.f;
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
    todo -= t_end - tile;
    if (todo > 0) {
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
  if (gave_up) {   // count it, and let the copies that may still come land before the memory is another's
    if (lane == 0) record_device_error(a.timeouts);   // null where the device has no counter
    for (int i = 0; i < L::slots; ++i) {
      mbar_wait(bar + slot, parity, &never, kWaitNs / 16);
      if (++slot == L::slots) {
        slot = 0;
        parity ^= 1;
      }
    }
  }
  if (!early) return;
  // The parts of the CTA's warps: those of one group follow one another.  A warp takes one head of one group at a time.
  __syncthreads();
  const Segment& own = segments[lane < 2 * kWarps ? lane : 0];
  const uint32_t there = __ballot_sync(0xffffffffu, lane < 2 * kWarps && own.part != nullptr);
  const bool opens = ((there >> lane) & 1u) && (own.begins || (there & ((1u << lane) - 1u)) == 0u);
  const uint32_t starts = __ballot_sync(0xffffffffu, opens);
  constexpr int kCols = D / 32;   // of a lane
  for (int item = warp; item < __popc(starts) * H; item += kWarps) {
    const int group = item / H, head = item - group * H;
    uint32_t rest = starts;
    for (int i = 0; i < group; ++i) rest &= rest - 1;
    const int first = __ffs(rest) - 1;
    const uint32_t later = rest & (rest - 1);   // the starts behind this one
    const uint32_t mine_of = there & ~((1u << first) - 1u) & (later ? (later & (0u - later)) - 1u : 0xffffffffu);
    // lane s has the part of segment s
    const bool has = (mine_of >> lane) & 1u;
    const float mi = has ? own.part[head] : __int_as_float(0xff800000), li = has ? own.part[H + head] : 0.f;
    float m = mi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float weight = has ? pow2(mi - (m == __int_as_float(0xff800000) ? 0.f : m)) : 0.f;
    const float l = warp_sum(li * weight);
    float acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
    for (uint32_t left = mine_of; left;) {   // four parts at a time
      float v[4][kCols], k[4];
      const int here = __popc(left) < 4 ? __popc(left) : 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = left ? __ffs(left) - 1 : first;
        k[q] = __shfl_sync(0xffffffffu, weight, i);
        left &= left - 1;
        const float* p = segments[i].part + 2 * H + head * D + kCols * lane;
        if (kCols == 4) {
          const float4 w = *reinterpret_cast<const float4*>(p);
          v[q][0] = w.x; v[q][1] = w.y; v[q][kCols - 2] = w.z; v[q][kCols - 1] = w.w;
        } else {
          const float2 w = *reinterpret_cast<const float2*>(p);
          v[q][0] = w.x; v[q][1] = w.y;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (q < here) acc[c] = fmaf(v[q][c], k[q], acc[c]);   // a part of weight 0 counts: its NaN stays one
    }
    const Segment& seg = segments[first];
    const int hk = seg.u / a.gtiles, hd = (seg.u - hk * a.gtiles) * H + head;
    if (seg.begins && segments[31 - __clz(mine_of)].ends) {
      if (hd >= a.G) continue;
      const size_t at = static_cast<size_t>(seg.b) * a.Hq + static_cast<size_t>(hk) * a.G + hd;
      const float f = l == 0.f ? 0.f : gate_of(a, seg.b, hk * a.G + hd) / l;
#pragma unroll
      for (int c = 0; c < kCols; c += 2)
        store2(static_cast<TO*>(a.out) + at * D + kCols * lane + c, acc[c] * f, acc[c + 1] * f);
      if (a.lse && lane == 0) a.lse[at] = (m + log2f(l)) * kLn2;
    } else {
      float* part = a.parts + (static_cast<size_t>(blockIdx.x) * 2 + (first == 0 ? 0 : 1)) * part_floats<D, HT>();
      if (lane == 0) {
        part[head] = m;
        part[H + head] = l;
      }
#pragma unroll
      for (int c = 0; c < kCols; c += 2) store2(part + 2 * H + head * D + kCols * lane + c, acc[c], acc[c + 1]);
    }
  }
}

// Joins the parts of the groups that were cut and writes the rows of empty sequences.
template <int D, int HT, typename TO>
__global__ void __launch_bounds__(kJoinThreads, 3) join_kernel(AttnArgs a) {
  constexpr int H = 8 * HT, kJoinWarps = kJoinThreads / 32, kLanes = D / 4, kRows = kJoinThreads / kLanes;
  __shared__ long long sums[2][kJoinWarps];
  __shared__ float red_m[kRows], red_l[kRows];
  __shared__ float4 red[kRows][kLanes];
  // D / 4 lanes have one head and every `ways`-th of its parts
  const int per_group = (a.G + (1 << a.together) - 1) >> a.together;
  const int ways_log2 = (kRows == 8 ? 3 : 4) - a.together, ways = 1 << ways_log2;
  const int group = blockIdx.x / per_group, b = group / a.Hkv, hk = group - b * a.Hkv;
  const int col = threadIdx.x % kLanes, row = threadIdx.x / kLanes, first = row & (ways - 1);
  const int in_group = ((blockIdx.x - group * per_group) << a.together) + (row >> ways_log2);   // heads of a block share a tile
  const int gt = in_group / H, head = in_group - gt * H, hq = hk * a.G + in_group;
  const bool real = in_group < a.G;
  // the tiles of all sequences, and of those before this one
  const int units = a.Hkv * a.gtiles, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long total = 0, before = 0;
  for (int i = threadIdx.x; i < a.B; i += kJoinThreads) {
    const int t = tiles_of(seq_len<true>(a, i));
    total += t;
    if (i < b) before += t;
  }
  const int nt = tiles_of(seq_len<true>(a, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    sums[0][warp] = total;
    sums[1][warp] = before;
  }
  __syncthreads();
  total = before = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    total += sums[0][w];
    before += sums[1][w];
  }
  total *= units;
  const long long p0 = before * units + static_cast<long long>(hk * a.gtiles + gt) * nt;
  constexpr int kWarps = warps_of<HT>();
  int w0 = 0, parts = 0, first_slot = 0;
  if (nt > 0) {
    const Pieces pieces(total, a.ctas * kWarps);
    const bool early = joined_early(a, pieces);
    const int x = pieces.owner(p0), y = pieces.owner(p0 + nt - 1);
    w0 = early ? x / kWarps : x;
    parts = (early ? y / kWarps : y) - w0 + 1;
    first_slot = pieces.start(early ? w0 * kWarps : w0) == p0 ? 0 : 1;
  }
  TO* out = static_cast<TO*>(a.out) + (static_cast<size_t>(b) * a.Hq + hq) * D;
  const float* base = a.parts + static_cast<size_t>(w0) * 2 * part_floats<D, HT>();
  auto part_of = [&](int i) { return base + static_cast<size_t>(2 * i + (i == 0 ? first_slot : 0)) * part_floats<D, HT>(); };
  // The first kernel's grid is done, and its writes are visible, behind this line; every block passes it, for what
  // comes next begins when this grid ends.  It is not let in early: the blocks of the next step's first kernel fill the
  // machine, and came to lie unevenly beside these (64 to 77 us a call at 286k E4M3 tokens).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (nt == 0) {   // the first kernel does not touch these rows
    if (real && first == 0) {
      store2(out + 4 * col, 0.f, 0.f);
      store2(out + 4 * col + 2, 0.f, 0.f);
      if (a.lse && col == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = __int_as_float(0xff800000);
    }
    return;
  }
  if (parts == 1) return;   // written whole
  constexpr int kBatch = 8;   // parts in flight, with a running maximum
  float m = __int_as_float(0xff800000), l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 < parts; i0 += ways * kBatch) {
    float mi[kBatch], li[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + q * ways;
      mi[q] = __int_as_float(0xff800000);
      if (i < parts) {
        const float* p = part_of(i);
        mi[q] = __ldcg(p + head);
        li[q] = __ldcg(p + H + head);
        v[q] = __ldcg(reinterpret_cast<const float4*>(p + 2 * H + head * D) + col);
      }
    }
    float top = m;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) top = fmaxf(top, mi[q]);
    const float zero = top == __int_as_float(0xff800000) ? 0.f : top;
    const float keep = exp2f(m - zero);
    l *= keep;
    acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
    m = top;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (i0 + q * ways < parts) {
        const float k = exp2f(mi[q] - zero);
        l = fmaf(li[q], k, l);
        acc.x = fmaf(v[q].x, k, acc.x);
        acc.y = fmaf(v[q].y, k, acc.y);
        acc.z = fmaf(v[q].z, k, acc.z);
        acc.w = fmaf(v[q].w, k, acc.w);
      }
    }
  }
  if (ways > 1) {
    red[row][col] = acc;
    if (col == 0) {
      red_m[row] = m;
      red_l[row] = l;
    }
    __syncthreads();
    if (first != 0) return;
    for (int r = row + 1; r < row + ways && r - row < parts; ++r) {
      const float other = red_m[r], top = fmaxf(m, other), zero = top == __int_as_float(0xff800000) ? 0.f : top;
      const float k0 = exp2f(m - zero), k1 = exp2f(other - zero);
      const float4 v = red[r][col];
      m = top;
      l = l * k0 + red_l[r] * k1;
      acc.x = acc.x * k0 + v.x * k1;
      acc.y = acc.y * k0 + v.y * k1;
      acc.z = acc.z * k0 + v.z * k1;
      acc.w = acc.w * k0 + v.w * k1;
    }
  }
  if (!real) return;
  const float f = l == 0.f ? 0.f : gate_of(a, b, hq) / l;
  store2(out + 4 * col, acc.x * f, acc.y * f);
  store2(out + 4 * col + 2, acc.z * f, acc.w * f);
  if (a.lse && col == 0) a.lse[static_cast<size_t>(b) * a.Hq + hq] = (m + log2f(l)) * kLn2;
}

template <int D, bool FP8, int HT, typename TO>
zmoe_status launch(AttnArgs a, cudaStream_t s) {
  using L = Lay<D, FP8, HT>;
  a.ctas = num_sms();
  // the cache as rows of one or two lines of 128 bytes (two rows of an 8-bit cache of 64 columns are a line)
  const cuuint32_t lines = L::row == 256 ? 2 : 1, tall = L::row == 64 ? 8 : 16;
  const cuuint64_t rows = static_cast<cuuint64_t>(a.n_pages) * a.Hkv * a.page_size * tall / 16;
  const cuuint64_t dims[3] = {128, lines, rows}, stride[2] = {128, 128 * lines};
  const cuuint32_t box[3] = {128, lines, tall};
  CUtensorMap km, vm;
  if (!encode_map(&km, a.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, stride, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map(&vm, a.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, stride, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return fail(ZMOE_ERR_CUDA, "zmoe_paged_attention: the cache's tensor map cannot be made");
  if (cudaFuncSetAttribute(attn_kernel<D, FP8, HT, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem) != cudaSuccess)
    return check_launch("zmoe_paged_attention: shared memory attribute");
  const zmoe_status st = launch_behind("zmoe_paged_attention", attn_kernel<D, FP8, HT, TO>, dim3(a.ctas),
                                       dim3(32 * L::warps), L::smem, s, 1, km, vm, a);
  if (st != ZMOE_OK) return st;
  // A block a head, unless they are more than run at once: then it takes up to 8 heads of a group.
  a.together = 0;
  auto join_blocks = [&]() { return static_cast<long long>(a.B) * a.Hkv * ((a.G + (1 << a.together) - 1) >> a.together); };
  while (join_blocks() > 3LL * num_sms() && a.together < 3 && (1 << a.together) < a.G) ++a.together;
  return launch_behind("zmoe_paged_attention (join)", join_kernel<D, HT, TO>, dim3(static_cast<unsigned>(join_blocks())),
                       dim3(kJoinThreads), 0, s, 1, a);
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
  return static_cast<size_t>(num_sms()) * kMaxWarps * 2 * H * (D + 2) * 4;
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
  ZMOE_REQUIRE(static_cast<unsigned long long>(n_pages) * Hkv * page_size < 0x7fffffffULL,
               "zmoe_paged_attention: n_pages * Hkv * page_size overflows int32");
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
  a.timeouts = device_timeout_counter();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = out_dtype == ZMOE_BF16;
  if (kv_dtype == ZMOE_E4M3) return D == 64 ? launch_out<64, true>(a, bf, s) : launch_out<128, true>(a, bf, s);
  return D == 64 ? launch_out<64, false>(a, bf, s) : launch_out<128, false>(a, bf, s);
}

}  // extern "C"
