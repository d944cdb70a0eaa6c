// decode8.cu -- single-token attention over 8-bit tile records and the FP32 window.
//
//   split kernel   grid (item, KV head, sequence). A tile item owns `span` consecutive
//                  tiles of one KV head; a window item owns a run of window rows. It
//                  writes the item's softmax maximum m, sum l and value accumulator
//                  (in units of 2^m) to the workspace.
//   merge kernel   grid (query head | KV head and run of tiles, sequence): joins the
//                  items of a head, sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i, and,
//                  on request, adds each tile's weight over the heads of its group.
//
// All G <= 8 query heads of a KV head share one pass over its records. Both products
// run on mma.sync m16n8k16 (fp16 in, fp32 out) with the codes as the B operand: a code
// is exact in fp16, so only the other operand is split. The query rows, scaled by a
// power of two each, and the weighted probabilities enter as pairs hi + lo (22 bits) in
// the 16 rows of A: head g's hi part in row g and its lo part in row g + 8. The two
// parts of a result then lie in registers of one lane and are added there, and the
// accumulator layout of the scores is a permutation of the A layout of the second product.
//   s_t = (q . code_t) * (kscale_t scale),   O += (2^(s_t - m) vscale_t) code_t
// A scale is constant over 16 tokens, so it multiplies scores and probabilities, never codes.
// The weighted probabilities have a reference exponent u of their own (their running
// maximum), so that any ratio between the value scales keeps its 22 bits.
//
// Records arrive by bulk copies into a ring of slots. Their code order is
// made for this kernel: a warp's 16-byte reads cover 512 consecutive bytes, and what a
// lane reads is what it needs of the B fragments of four products, up to an order of the
// summed index (channels, or tokens) that both operands share.
//
// A CTA's warps split a tile's tokens for the scores and its channels for the values, with one exchange of
// row maxima and one of probabilities per step of one or two tiles through shared memory.
//
// HBM bounds it in batches: 32 ragged sequences of up to 32k tokens, head_dim 256, 1.37 GB in 218 us
// (6.3 TB/s, 93% of the measured copy rate; one CTA per SM with whole records in its stages took 311);
// 4 of 64k tokens, head_dim 128, 0.54 GB in 94 us (84%), where the instructions per code (conversion,
// products, exchanges: 1.6 per cycle and SM) take as long as the copy. One sequence of 16k tokens, 34 MB,
// takes 12.5 us against a floor of 5: an almost empty call takes 7.6 (launch, count, table, copy, exchanges,
// merge: a chain of latencies), then HBM counts. One cluster per head that joins its items itself, instead of
// the merge kernel, took 8.9 us where two kernels take 8.2.
//
// The same kernels serve chunks of a few positions (CHUNK): eight (position, head) rows to a CTA, each of
// which sees the cache up to its own position.
#include "cache8.cuh"
#include "join.cuh"

namespace kvarn {
namespace {

constexpr float kNone = -3.0e38f;  // reference exponent before the first tile
constexpr int kPRow = 576;          // bytes per head of the probability buffer (4 bytes x 2 parts x 64 pairs + pad)
constexpr float kHead = 14.f;       // weighted probabilities reach 2^14: lo parts stay normal fp16 numbers

template <int D_>
struct D8 {
  static constexpr int D = D_;
  static constexpr int NW = 8;                   // warps per CTA
  static constexpr int NTHR = 32 * NW;
  static constexpr int NT = 16 / NW;             // 8-token column tiles of the scores per warp
  // The values are split over the warps by channels, and where that leaves a warp one column tile of 8, by
  // the halves of a tile's tokens too: what a warp reads of the probabilities is then read for more channels
  // (24 ragged sequences, seven heads to a group: 60.0 -> 56.6 us).
  static constexpr int TS = D == 64 ? 2 : 1;
  static constexpr int NC = D / 8 / (NW / TS);   // column tiles of the values per warp
  static constexpr int NCW = D / 8 / NW;         // the same for a window's values
  static constexpr int NJ = D / 64;              // 64-channel runs
  // A record arrives as two copies, K codes with the scales behind them, and V codes, each in a slot of a
  // ring: two (four, at head_dim 64) CTAs per SM have some 100 KB in flight or in use, and a CTA's
  // exchanges are covered by the other's work
  static constexpr int HALF = kTile * D;         // bytes of K or of V codes
  static constexpr int SLOT = HALF + 128;
  // Tiles of a step: two halve the exchanges (4 of 64k tokens, head_dim 128: 97.1 -> 94.4 us; 5 ragged ones,
  // head_dim 64: 21.1 -> 20.5); at head_dim 256 neither slots nor registers are left for it.
  static constexpr int TP = D <= 128 ? 2 : 1;
  static constexpr int SLOTS = D == 256 ? 3 : D == 64 ? 5 : 6;
  static constexpr int CTAS = D == 64 ? 4 : 2;   // resident per SM
  // The tensor core drops what falls below a sum's last bit. Where registers allow, a score is two sums
  // and a step's values a sum of their own, joined with rounding (at head_dim 256 they spill: 224 us of
  // batched decode become 245; at 64 they cost 5% and gain nothing).
  static constexpr bool FRESH = D == 128;
  static constexpr int WROWS = 8 * NW;           // window rows per window item
  static constexpr int OFF_P = SLOTS * SLOT;
  static constexpr int OFF_MX = OFF_P + TP * 8 * kPRow;              // float2 [8][NW]: (max s, max s + log2 vscale)
  static constexpr int OFF_L = OFF_MX + 8 * NW * 8;             // float [TP][NW][8]
  static constexpr int OFF_BAR = OFF_L + TP * 8 * NW * 4;
  static constexpr int OFF_FLG = OFF_BAR + 8 * SLOTS;         // int: a wait ran out or a record was refused
  static constexpr int SMEM = (OFF_FLG + 8 + 127) / 128 * 128;
  static_assert(SLOTS > TP && SLOTS + TP <= 4 * TP, "a step's requests belong to it and to the next");
  static_assert(SLOT % 128 == 0 && OFF_P % 128 == 0, "alignment");
  static_assert(8 * (WROWS + 4) * 4 <= 8 * kPRow, "window probabilities fit");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, both brought to the 11 bits that a tf32 operand is read with: within 2^-21 of x. hi is rounded by an
// addition to its bits. For lo, from which the tensor core cuts the rest, a product does it (0.36 to 0.72 of the
// last kept bit is added before the cut), because of an infinity or a NaN lo has to stay NaN, so that every score it
// enters is NaN whatever the signs: NaN is the largest int, an addition to its bits would wrap to -0.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  const uint32_t u = __float_as_uint(x), r = u + 0x1000u;
  hi = ((r & 0x7F800000u) == 0x7F800000u ? u : r) & 0xFFFFE000u;  // (not up to infinity)
  lo = __float_as_uint((x - __uint_as_float(hi)) * (1.f + 0x1.7p-12f));
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, shfl_xor(v, 1));
  return fmaxf(v, shfl_xor(v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += shfl_xor(v, 1);
  return v + shfl_xor(v, 2);
}

// Sum over the CTA's warps of a quad-reduced row value l of head g (lanes with q == 0 hold it).
template <int NW>
__device__ __forceinline__ float cta_row_sum(float l, float* buf, int warp, int g, int q) {
  __syncthreads();
  if (q == 0) buf[warp * 8 + g] = l;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += buf[w * 8 + g];
  return s;
}

struct Split8Args {
  Decode8Args a;
  float2* ml;      // [B][Hq][items]
  float* acc;      // [B][Hq][items][D]
  float2* tile_ml; // [B][Hkv][max_tiles][8], or NULL
  int span, tile_items, items;
  // a chunk of positions (CHUNK): B positions of one sequence instead of B sequences
  int64_t pos0;
  int n_tiles, win_start, win_len;
};

// Score row g of a CTA: with CHUNK the (position, head) pairs of a KV head, eight per CTA, are rows of one
// sequence that see the cache up to their own position; otherwise the G heads of sequence blockIdx.z.
struct Row8 {
  bool valid;
  int64_t index;  // among the [B][Hq] rows of queries and outputs
  int64_t seen;   // cached tokens that the row sees
};
template <bool CHUNK>
__device__ __forceinline__ Row8 row8(const Split8Args& s, int kvh, int g) {
  const Decode8Args& a = s.a;
  if constexpr (CHUNK) {
    const int r = 8 * blockIdx.z + g, i = r / a.G;
    const bool valid = i < a.B;
    return Row8{valid, valid ? (int64_t)i * a.Hq + (int64_t)kvh * a.G + r % a.G : 0, valid ? s.pos0 + i + 1 : 0};
  } else {
    return Row8{g < a.G, (int64_t)blockIdx.z * a.Hq + (int64_t)kvh * a.G + min(g, a.G - 1), INT64_MAX};
  }
}

// A run of window rows: fp32 rows against fp32 queries and probabilities, every operand a
// pair of tf32 numbers. A row with a NaN or an infinity counts as NaN scores and zero values.
template <int D, bool CHUNK>
__device__ __forceinline__ void window_item(const Split8Args& s, unsigned char* smem, int item, int kvh) {
  using C = D8<D>;
  const Decode8Args& a = s.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  float* P = reinterpret_cast<float*>(smem + C::OFF_P);
  float2* mx = reinterpret_cast<float2*>(smem + C::OFF_MX);
  volatile int* dead = reinterpret_cast<volatile int*>(smem);  // [WROWS]
  constexpr int PS = C::WROWS + 4;
  const int b = CHUNK ? 0 : blockIdx.z;
  const Row8 me = row8<CHUNK>(s, kvh, g);
  const int wlen = CHUNK ? s.win_len : min(max(a.win_len[b], 0), a.win_cap);
  const int r0 = C::WROWS * (item - s.tile_items);
  const int n = min(C::WROWS, wlen - r0);
  pdl_trigger();
  if (n <= 0) {
    if (tid < 8) {
      const Row8 r = row8<CHUNK>(s, kvh, tid);
      if (r.valid) s.ml[r.index * s.items + item] = make_float2(-INFINITY, 0.f);
    }
    return;
  }
  const int start = CHUNK ? s.win_start : ((a.win_start[b] % a.win_cap) + a.win_cap) % a.win_cap;
  const int64_t head = ((int64_t)b * a.Hkv + kvh) * a.win_cap;
  auto row = [&](int t) { return (head + ((int64_t)start + r0 + t) % a.win_cap) * (int64_t)D; };
  // rows of this item that score row g sees
  const int seen = CHUNK ? (int)max((int64_t)0, min((int64_t)n, me.seen - (int64_t)128 * s.n_tiles - r0)) : n;
  if (tid < C::WROWS) dead[tid] = 0;
  __syncthreads();
  // the values this warp's channels need: under way while the scores are formed, where registers allow
  float v[C::NW][C::NCW][2];
  auto load_values = [&] {
#pragma unroll
    for (int k = 0; k < C::NW; ++k) {
      const int t0 = 8 * k + q, t1 = t0 + 4;
      const float* v0 = a.win_v + (t0 < n ? row(t0) : 0) + 8 * C::NCW * warp + g;
      const float* v1 = a.win_v + (t1 < n ? row(t1) : 0) + 8 * C::NCW * warp + g;
#pragma unroll
      for (int c = 0; c < C::NCW; ++c) {
        v[k][c][0] = t0 < n ? v0[8 * c] : 0.f;
        v[k][c][1] = t1 < n ? v1[8 * c] : 0.f;
      }
    }
  };
  if constexpr (D <= 128) load_values();
  const bool have = 8 * warp + g < n;
  const float* kr = a.win_k + (have ? row(8 * warp + g) : 0) + 4 * q;
  const int64_t qrow = me.index * D + 4 * q;
  // sums of their own for the parts of K and for odd and even steps: the tensor core cuts off what falls below
  // a sum's last bit, and no product waits for the one before
  float sh[2][4] = {}, sl[2][4] = {};
  // loads of K and of the queries under way together, beside those of V where they come first (3 tiles and a
  // window, head_dim 128: 7.6 us; all of them at once 8.2, in the order of use 8.9)
  constexpr int RUN = D == 64 ? 2 : D == 128 ? 4 : 8;
#pragma unroll 1
  for (int m0 = 0; m0 < D / 16; m0 += RUN) {
    float4 kx[RUN], qx[RUN];
#pragma unroll
    for (int m = 0; m < RUN; ++m) {
      kx[m] = have ? *reinterpret_cast<const float4*>(kr + 16 * (m0 + m)) : make_float4(0.f, 0.f, 0.f, 0.f);
      qx[m] = me.valid ? io_ld4(a.q, a.io, qrow + 16 * (m0 + m)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int m = 0; m < RUN; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t qa[4], kh[2], kl[2];
        split_tf32(h ? qx[m].z : qx[m].x, qa[0], qa[1]);
        split_tf32(h ? qx[m].w : qx[m].y, qa[2], qa[3]);
        split_tf32(h ? kx[m].z : kx[m].x, kh[0], kl[0]);
        split_tf32(h ? kx[m].w : kx[m].y, kh[1], kl[1]);
        mma_tf32(sh[h], qa, kh[0], kh[1]);
        mma_tf32(sl[h], qa, kl[0], kl[1]);
      }
  }
  if constexpr (D == 256) load_values();
#pragma unroll
  for (int k = 0; k < C::NW; ++k)
#pragma unroll
    for (int c = 0; c < C::NCW; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (!isfinite(v[k][c][h])) {
          dead[8 * k + q + 4 * h] = 1;
          v[k][c][h] = 0.f;
        }
  float sc[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    sc[e] = ((sl[0][e] + sl[1][e]) + ((sh[0][e + 2] + sl[0][e + 2]) + (sh[1][e + 2] + sl[1][e + 2]))) +
            (sh[0][e] + sh[1][e]);
  const int t0 = 8 * warp + 2 * q;
  __syncthreads();  // dead rows are known
  const float s0 = t0 < seen ? (dead[t0] ? NAN : sc[0] * a.scale) : -INFINITY;
  const float s1 = t0 + 1 < seen ? (dead[t0 + 1] ? NAN : sc[1] * a.scale) : -INFINITY;
  const float mw = quad_max(fmaxf(s0, s1));
  if (q == 0) mx[g * C::NW + warp].x = mw;
  __syncthreads();
  float M = kNone;
#pragma unroll
  for (int w = 0; w < C::NW; ++w) M = fmaxf(M, mx[g * C::NW + w].x);
  const float p0 = t0 < seen ? fast_ex2(s0 - M) : 0.f, p1 = t0 + 1 < seen ? fast_ex2(s1 - M) : 0.f;
  *reinterpret_cast<float2*>(P + g * PS + t0) = make_float2(p0, p1);
  const float l = cta_row_sum<C::NW>(quad_sum(p0 + p1), reinterpret_cast<float*>(smem + C::OFF_L), warp, g, q);
  float o[C::NCW][4] = {}, olo[C::NCW][4] = {};
  float (&ol)[C::NCW][4] = D <= 128 ? olo : o;
#pragma unroll
  for (int k = 0; k < C::NW; ++k) {
    uint32_t pa[4];
    split_tf32(P[g * PS + 8 * k + q], pa[0], pa[1]);
    split_tf32(P[g * PS + 8 * k + q + 4], pa[2], pa[3]);
#pragma unroll
    for (int c = 0; c < C::NCW; ++c) {
      uint32_t vh[2], vl[2];
      split_tf32(v[k][c][0], vh[0], vl[0]);
      split_tf32(v[k][c][1], vh[1], vl[1]);
      mma_tf32(o[c], pa, vh[0], vh[1]);
      mma_tf32(ol[c], pa, vl[0], vl[1]);
    }
  }
  if constexpr (D <= 128) {
#pragma unroll
    for (int c = 0; c < C::NCW; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[c][r] += olo[c][r];
  }
  if (me.valid) {
    const int64_t part = me.index * s.items + item;
    float* dst = s.acc + part * D + 8 * C::NCW * warp + 2 * q;
#pragma unroll
    for (int c = 0; c < C::NCW; ++c)
      *reinterpret_cast<float2*>(dst + 8 * c) = make_float2(o[c][0] + o[c][2], o[c][1] + o[c][3]);
    if (warp == 0 && q == 0) s.ml[part] = make_float2(M, l);
  }
}

template <int D, int F, bool CHUNK>
__global__ void __launch_bounds__(D8<D>::NTHR, D8<D>::CTAS) split8_kernel(const Split8Args s) {
  using C = D8<D>;
  using R = Rec8<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  const Decode8Args& a = s.a;
  const int item = blockIdx.x, kvh = blockIdx.y, b = CHUNK ? 0 : blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  if (item >= s.tile_items) {
    pdl_wait();
    window_item<D, CHUNK>(s, smem, item, kvh);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLG);
  // with prefetch, the records (which, by the caller's guarantee, nothing still running
  // writes) are requested before the previous kernel on the stream is waited for
  const bool early = a.flags & KVARN_LAUNCH_PREFETCH;
  if (!early) pdl_wait();
  const int first = item * s.span;
  const int64_t* table = a.tile_table + ((int64_t)b * a.Hkv + kvh) * a.max_tiles + first;
  // The requesting thread holds the table's entries of two steps: the first ones are read beside the count, not
  // after it (all lie inside the table), the others a step before they are needed.
  constexpr int TP = C::TP;
  int64_t entry[2][TP] = {};
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < 2 * TP; ++k)
      if (first + k < (CHUNK ? s.n_tiles : a.max_tiles)) entry[k / TP][k % TP] = __ldcg(table + k);
  }
  const int n_tiles = CHUNK ? s.n_tiles : min(max(a.n_tiles[b], 0), a.max_tiles);
  const int nt = min(max(n_tiles - first, 0), s.span);
  if (nt == 0) {
    if (early) pdl_wait();
    pdl_trigger();
    if (tid < 8) {
      const Row8 r = row8<CHUNK>(s, kvh, tid);
      if (r.valid) s.ml[r.index * s.items + item] = make_float2(-INFINITY, 0.f);
    }
    return;
  }
  // one thread: copy n of the item (K of a step's tiles, then V) into its slot; off: the tile's entry
  auto request = [&](int n, int64_t off) {
    const int tile = n / (2 * TP) * TP + n % TP;
    if (n < 0 || tile >= nt) return;
    const bool is_v = n % (2 * TP) >= TP;
    uint64_t* br = bar + n % C::SLOTS;
    unsigned char* dst = smem + (n % C::SLOTS) * C::SLOT;
    if ((off & 15) || off < 0 || off > a.tiles_bytes - R::kBytes) {
      // a record that is not read: zero codes under scales of NaN, which only rows that see it meet
      report(a.err, KVARN_DEVERR_RECORD);
      for (int k = 0; k < C::HALF; k += 16) *reinterpret_cast<uint4*>(dst + k) = make_uint4(0, 0, 0, 0);
      for (int k = 0; k < 2 * kGrps; ++k) reinterpret_cast<float*>(dst + C::HALF)[k] = NAN;
      mbar_arrive1(br);
      return;
    }
    if (is_v) {
      mbar_arrive_tx(br, C::HALF);
      bulk_in(dst, a.tiles + off + R::kVCodes, C::HALF, br);
    } else {
      mbar_arrive_tx(br, C::HALF + 8 * kGrps);
      bulk_in(dst, a.tiles + off + R::kKCodes, C::HALF, br);
      bulk_in(dst + C::HALF, a.tiles + off + R::kKScale, 8 * kGrps, br);
    }
  };
  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) mbar_init_n(bar + i, 1);
    mbar_fence_init();
    *flag = 0;
#pragma unroll
    for (int i = 0; i < C::SLOTS; ++i) request(i, entry[i / (2 * TP)][i % TP]);
  }
  if (early) pdl_wait();
  pdl_trigger();

  // A fragments of the query: head g's row, channels 64 j + 16 q + 4 r + {0, 1} and {2, 3}
  // of product (j, r); hi in the registers of row g, lo in those of row g + 8
  uint32_t qa[4 * C::NJ][4];
  float c1;
  [[maybe_unused]] int64_t seen = 0;  // cached tokens that row g sees (CHUNK)
  {
    const Row8 me = row8<CHUNK>(s, kvh, g);
    seen = me.seen;
    float x[C::NJ][16];
    const int64_t qrow = me.index * D + 16 * q;
    float mxq = 0.f;
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 v = me.valid ? io_ld4(a.q, a.io, qrow + 64 * j + 4 * r) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[j][4 * r] = v.x; x[j][4 * r + 1] = v.y; x[j][4 * r + 2] = v.z; x[j][4 * r + 3] = v.w;
        mxq = fmaxf(fmaxf(mxq, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
      }
    const float p2 = pow2_to(quad_max(mxq), 10);
    c1 = a.scale * pow2_inverse(p2);
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        split_pair(x[j][4 * r] * p2, x[j][4 * r + 1] * p2, qa[4 * j + r][0], qa[4 * j + r][1]);
        split_pair(x[j][4 * r + 2] * p2, x[j][4 * r + 3] * p2, qa[4 * j + r][2], qa[4 * j + r][3]);
      }
  }
  float2* mx = reinterpret_cast<float2*>(smem + C::OFF_MX);
  float* lbuf = reinterpret_cast<float*>(smem + C::OFF_L);
  unsigned char* P = smem + C::OFF_P;
  __syncthreads();  // barriers initialised

  float M = kNone, U = kNone, l = 0.f;
  float o[C::NC][4] = {};
  float sc[TP][C::NT][2];
  float vs[TP];
  bool ok = true;
  const int grp = (warp * C::NT) >> 1;  // scale entry of this warp's tokens
  const int cw = warp % (C::NW / C::TS);  // place among the channels

  auto landed = [&](int n) { return mbar_wait8(bar + n % C::SLOTS, (uint32_t)(n / C::SLOTS) & 1u, a.err); };
  // scores of step j (tiles TP j ..): of each tile the tokens 8 NT warp .., and their row maxima
  auto scores = [&](int j) {
    float mw = -INFINITY, uw = -INFINITY;
#pragma unroll
    for (int x = 0; x < TP; ++x) {
      if (TP > 1 && x > 0 && TP * j + x >= nt) {  // an odd item's last step
#pragma unroll
        for (int t = 0; t < C::NT; ++t) sc[x][t][0] = sc[x][t][1] = -INFINITY;
        vs[x] = 0.f;
        break;
      }
      const int n = 2 * TP * j + x;
      ok &= landed(n);
      const unsigned char* rec = smem + (n % C::SLOTS) * C::SLOT;
      const float kc = reinterpret_cast<const float*>(rec + C::HALF)[grp] * c1;
      vs[x] = reinterpret_cast<const float*>(rec + C::HALF)[kGrps + grp];
      float mt = -INFINITY;
#pragma unroll
      for (int t = 0; t < C::NT; ++t) {
        float c[4] = {0.f, 0.f, 0.f, 0.f}, d[4] = {0.f, 0.f, 0.f, 0.f};
        float (&e)[4] = C::FRESH ? d : c;
#pragma unroll
        for (int k = 0; k < C::NJ; ++k) {
          const uint4 w = *reinterpret_cast<const uint4*>(rec +
                                                          ((warp * C::NT + t) * C::NJ + k) * 512 + lane * 16);
          uint32_t b0, b1;
          codes_to_half<F>(w.x, b0, b1); mma_f16(c, qa[4 * k], b0, b1);
          codes_to_half<F>(w.y, b0, b1); mma_f16(c, qa[4 * k + 1], b0, b1);
          codes_to_half<F>(w.z, b0, b1); mma_f16(e, qa[4 * k + 2], b0, b1);
          codes_to_half<F>(w.w, b0, b1); mma_f16(e, qa[4 * k + 3], b0, b1);
        }
        sc[x][t][0] = ((c[0] + d[0]) + (c[2] + d[2])) * kc;
        sc[x][t][1] = ((c[1] + d[1]) + (c[3] + d[3])) * kc;
        if constexpr (CHUNK) {
          const int64_t pos = (int64_t)128 * (first + TP * j + x) + 8 * (warp * C::NT + t) + 2 * q;
          if (pos >= seen) sc[x][t][0] = -INFINITY;
          if (pos + 1 >= seen) sc[x][t][1] = -INFINITY;
        }
        mt = fmaxf(mt, fmaxf(sc[x][t][0], sc[x][t][1]));
      }
      mw = fmaxf(mw, mt);
      uw = fmaxf(uw, mt + fast_lg2(vs[x]));
    }
    mw = quad_max(mw);
    if (TP > 1) uw = quad_max(uw);
    if (q == 0) mx[g * C::NW + warp] = make_float2(mw, TP > 1 ? uw : mw + fast_lg2(vs[0]));
  };

  const int n_steps = (nt + TP - 1) / TP;
  scores(0);
  for (int j = 0; j < n_steps; ++j) {
    __syncthreads();  // row maxima of step j are in; step j - 1 and its probabilities are used up
    if (tid == 0) {   // the slots of V of step j - 1 and of K of step j are free
#pragma unroll
      for (int n = -TP; n < TP; ++n)  // (what they are filled with belongs to step j or j + 1)
        if (j > 0 || n >= 0) request(2 * TP * j + n + C::SLOTS, entry[(n + C::SLOTS) / (2 * TP)][(n + C::SLOTS) % TP]);
#pragma unroll
      for (int k = 0; k < TP; ++k) {
        entry[0][k] = entry[1][k];
        if (TP * (j + 2) + k < nt) entry[1][k] = table[TP * (j + 2) + k];
      }
    }
    float Mn = M, Un = U;
#pragma unroll
    for (int w = 0; w < C::NW; w += 2) {
      const float4 v = *reinterpret_cast<const float4*>(mx + g * C::NW + w);
      Mn = fmaxf(Mn, fmaxf(v.x, v.z));
      Un = fmaxf(Un, fmaxf(v.y, v.w));
    }
    const float al = fast_ex2(M - Mn), ao = fast_ex2(U - Un);
    [[maybe_unused]] const bool moved = Un != U;
    M = Mn;
    U = Un;
    // weight of a value code: probability * scale, in units of 2^(U - kHead); a factor past the
    // range belongs to probabilities below 2^-100
    const float fm = fast_ex2(fminf(M - U + kHead, 126.f));
    float lt[TP];
#pragma unroll
    for (int x = 0; x < TP; ++x) {
      float fw = vs[x] * fm;
      if (fw > 1e30f) fw = 1e30f;
      lt[x] = 0.f;
#pragma unroll
      for (int t = 0; t < C::NT; ++t) {
        const float p0 = fast_ex2(sc[x][t][0] - M), p1 = fast_ex2(sc[x][t][1] - M);
        lt[x] += p0 + p1;
        uint32_t hi, lo;
        if constexpr (CHUNK)  // (a token that is not seen has weight 0, whatever its scale)
          split_pair(sc[x][t][0] == -INFINITY ? 0.f : p0 * fw, sc[x][t][1] == -INFINITY ? 0.f : p1 * fw, hi, lo);
        else
          split_pair(p0 * fw, p1 * fw, hi, lo);
        // tokens 8 n + 2 q, + 1 in the order the second product's A fragments are read
        const int n = warp * C::NT + t;
        *reinterpret_cast<uint2*>(P + (8 * x + g) * kPRow +
                                  (((n >> 3) * 4 + 2 * (n & 1) + (q >> 1)) * 4 + ((n & 7) >> 1)) * 16 + (q & 1) * 8) =
            make_uint2(hi, lo);
      }
    }
    l = fmaf(l, al, TP > 1 ? lt[0] + lt[TP - 1] : lt[0]);
    if (s.tile_ml) {
#pragma unroll
      for (int x = 0; x < TP; ++x) {
        lt[x] = quad_sum(lt[x]);
        if (q == 0) lbuf[(x * C::NW + warp) * 8 + g] = lt[x];
      }
    }
    __syncthreads();  // probabilities of step j are in
    if (s.tile_ml && warp < TP && TP * j + warp < nt && q == 0) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < C::NW; ++w) t += lbuf[(warp * C::NW + w) * 8 + g];
      s.tile_ml[(((int64_t)b * a.Hkv + kvh) * a.max_tiles + first + TP * j + warp) * 8 + g] = make_float2(M, t);
    }
    float fresh[C::NC][4] = {};
    float (&ot)[C::NC][4] = C::FRESH ? fresh : o;
    if (!C::FRESH && __any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int c = 0; c < C::NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[c][r] *= ao;
    }
#pragma unroll
    for (int x = 0; x < TP; ++x) {
      if (TP > 1 && x > 0 && TP * j + x >= nt) break;
      const int n = 2 * TP * j + TP + x;
      ok &= landed(n);
      const unsigned char* V = smem + (n % C::SLOTS) * C::SLOT;
#pragma unroll
      for (int h0 = 0; h0 < 2 / C::TS; ++h0) {
        const int h = C::TS == 2 ? warp / (C::NW / 2) : h0;
        uint4 w[C::NC];
#pragma unroll
        for (int c = 0; c < C::NC; ++c)
          w[c] = *reinterpret_cast<const uint4*>(V + ((cw * C::NC + c) * 2 + h) * 512 + lane * 16);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint4 f = *reinterpret_cast<const uint4*>(P + (8 * x + g) * kPRow + ((h * 4 + r) * 4 + q) * 16);
          const uint32_t pa[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int c = 0; c < C::NC; ++c) {
            uint32_t b0, b1;
            codes_to_half<F>((&w[c].x)[r], b0, b1);
            mma_f16(ot[c], pa, b0, b1);
          }
        }
      }
    }
    if constexpr (C::FRESH) {
#pragma unroll
      for (int c = 0; c < C::NC; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[c][r] = fmaf(o[c][r], ao, fresh[c][r]);
    }
    if (j + 1 < n_steps) scores(j + 1);
  }
  if (!ok) *flag = 1;
  l = cta_row_sum<C::NW>(quad_sum(l), lbuf, warp, g, q);  // its barriers also publish the flag
  const bool bad = *flag != 0;
  if (bad && tid == 0) {  // a copy whose wait ran out still writes to this CTA's memory: each is given as long again
    for (int n = max(0, 2 * TP * n_steps - C::SLOTS); n < 2 * TP * n_steps; ++n)
      if (n / (2 * TP) * TP + n % TP < nt) mbar_wait8(bar + n % C::SLOTS, (uint32_t)(n / C::SLOTS) & 1u, nullptr);
  }
  float r[C::NC][2];
#pragma unroll
  for (int c = 0; c < C::NC; ++c) {
    r[c][0] = o[c][0] + o[c][2];
    r[c][1] = o[c][1] + o[c][3];
  }
  if constexpr (C::TS == 2) {  // the two halves of the tokens meet in the first slot, which nothing needs any more
    float2* meet = reinterpret_cast<float2*>(smem) + (cw * C::NC) * 32 + lane;
    if (warp >= C::NW / 2) {
#pragma unroll
      for (int c = 0; c < C::NC; ++c) meet[32 * c] = make_float2(r[c][0], r[c][1]);
    }
    __syncthreads();
    if (warp >= C::NW / 2) return;
#pragma unroll
    for (int c = 0; c < C::NC; ++c) {
      r[c][0] += meet[32 * c].x;
      r[c][1] += meet[32 * c].y;
    }
  }
  const Row8 me = row8<CHUNK>(s, kvh, g);
  if (me.valid) {
    const int64_t part = me.index * s.items + item;
    const float f = fast_ex2(U - kHead - M);
    float* dst = s.acc + part * D + 8 * C::NC * cw + 2 * q;
#pragma unroll
    for (int c = 0; c < C::NC; ++c) *reinterpret_cast<float2*>(dst + 8 * c) = make_float2(r[c][0] * f, r[c][1] * f);
    if (warp == 0 && q == 0)
      s.ml[part] = bad ? make_float2(0.f, NAN) : make_float2(M, l);
  }
}

// Joins the items of query head blockIdx.x (blockIdx.x < Hq), or adds up the weights of 256 tiles
// of a KV head.
template <int D>
__global__ void __launch_bounds__(256) merge8_kernel(const Split8Args s, int mass_blocks) {
  const Decode8Args& a = s.a;
  const int b = blockIdx.y;
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x >= a.Hq) {
    const int kvh = ((int)blockIdx.x - a.Hq) / mass_blocks, run = ((int)blockIdx.x - a.Hq) % mass_blocks;
    const int64_t at = ((int64_t)b * a.Hkv + kvh) * a.max_tiles;
    join_masses<1>(s.ml + ((int64_t)b * a.Hq + kvh * a.G) * s.items, s.items, s.items, s.tile_ml + at * 8, a.G, run,
                   min(a.n_tiles[b], a.max_tiles), a.max_tiles, a.mass_in ? a.mass_in + at : nullptr, a.mass_out + at);
    return;
  }
  const int64_t row = (int64_t)b * a.Hq + blockIdx.x;
  join_items<D>(s.ml + row * s.items, s.acc + row * s.items * D, s.items, a.out, a.io, row);
}

template <int D, int F, bool CHUNK>
cudaError_t launch_d8(const Decode8Plan& p, Split8Args& s, void* ws, cudaStream_t st) {
  using C = D8<D>;
  const Decode8Args& a = s.a;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(split8_kernel<D, F, CHUNK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  unsigned char* w = static_cast<unsigned char*>(ws);
  s.ml = reinterpret_cast<float2*>(w);
  s.acc = reinterpret_cast<float*>(w + p.off_acc);
  s.tile_ml = a.mass_out ? reinterpret_cast<float2*>(w + p.off_tile) : nullptr;
  s.span = p.span;
  s.tile_items = p.tile_items;
  s.items = p.items;
  if (p.items > 0) {
    LaunchCfg L(dim3(p.items, a.Hkv, CHUNK ? (a.B * a.G + 7) / 8 : a.B), dim3(C::NTHR), C::SMEM, st, a.flags);
    e = cudaLaunchKernelEx(&L.cfg, split8_kernel<D, F, CHUNK>, s);
    if (e != cudaSuccess) return e;
  }
  const int mass_blocks = a.mass_out ? (a.max_tiles + 255) / 256 : 0;
  // the merge waits for the split kernel on the device, whatever the caller's flags
  LaunchCfg L(dim3(a.Hq + a.Hkv * mass_blocks, a.B), dim3(256), 0, st, a.flags | KVARN_LAUNCH_PDL);
  return cudaLaunchKernelEx(&L.cfg, merge8_kernel<D>, s, mass_blocks);
}

template <bool CHUNK>
cudaError_t launch_any(const Decode8Plan& p, Split8Args& s, void* ws, cudaStream_t st) {
  const bool e = s.a.format == KVARN_CODE8_E4M3;
  switch (s.a.D) {
    case 64: return e ? launch_d8<64, 1, CHUNK>(p, s, ws, st) : launch_d8<64, 0, CHUNK>(p, s, ws, st);
    case 128: return e ? launch_d8<128, 1, CHUNK>(p, s, ws, st) : launch_d8<128, 0, CHUNK>(p, s, ws, st);
    case 256: return e ? launch_d8<256, 1, CHUNK>(p, s, ws, st) : launch_d8<256, 0, CHUNK>(p, s, ws, st);
    default: return cudaErrorInvalidValue;
  }
}

// groups: CTAs that read a KV head's records; rows: query rows; seqs: sequences of lengths of their own.
void make_plan(int64_t groups, int64_t rows, int seqs, int D, int max_tiles, int win_rows, size_t tile_pairs,
               Decode8Plan* p) {
  const int ctas = D == 64 ? D8<64>::CTAS : D == 128 ? D8<128>::CTAS : D8<256>::CTAS;
  const int64_t slots = (int64_t)sm_count() * ctas;
  const int64_t work = groups * max_tiles;
  // Whole waves of resident CTAs, as long as an item has at most 16 tiles. Several sequences, whose
  // lengths differ as a rule, take two waves at least: a wave of items as long as the longest
  // sequence's leaves the SMs of the short ones idle (5 ragged sequences of up to 250 tiles, head_dim
  // 64: 24.7 -> 20.5 us; 8 equal ones of 256 tiles, head_dim 256: 92.9 -> 97.6 us).
  int64_t waves = (work + 16 * slots - 1) / (16 * slots);
  if (waves < (seqs > 1 ? 2 : 1)) waves = seqs > 1 ? 2 : 1;
  const int64_t span = (work + waves * slots - 1) / (waves * slots);
  p->span = (int)(span < 1 ? 1 : span);
  p->tile_items = (max_tiles + p->span - 1) / p->span;
  constexpr int kRows = D8<64>::WROWS;
  static_assert(kRows == D8<128>::WROWS && kRows == D8<256>::WROWS, "window rows per item");
  p->items = p->tile_items + (int)(((int64_t)win_rows + kRows - 1) / kRows);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p->off_acc = up((size_t)rows * p->items * sizeof(float2));
  p->off_tile = p->off_acc + up((size_t)rows * p->items * D * sizeof(float));
  p->ws_bytes = p->off_tile + up(tile_pairs * sizeof(float2));
}

}  // namespace

void decode8_plan(int B, int Hq, int Hkv, int D, int max_tiles, int win_capacity, Decode8Plan* p) {
  make_plan((int64_t)B * Hkv, (int64_t)B * Hq, B, D, max_tiles, win_capacity, (size_t)B * Hkv * max_tiles * 8, p);
}

cudaError_t launch_decode8(const Decode8Plan& p, const Decode8Args& a, void* ws, cudaStream_t st) {
  Split8Args s{};
  s.a = a;
  return launch_any<false>(p, s, ws, st);
}

// A few positions of one sequence, eight (position, head) rows of a KV head to a CTA.
void chunk8_plan(int C, int Hq, int Hkv, int D, int n_tiles, int win_len, Decode8Plan* p) {
  make_plan((int64_t)Hkv * ((C * (Hq / Hkv) + 7) / 8), (int64_t)C * Hq, 1, D, n_tiles, win_len, 0, p);
}

cudaError_t launch_chunk8(const Prefill8Args& a, int n_tiles, int win_len, cudaStream_t st) {
  // the plan that the workspace was counted for; fewer tiles are spread over as many items at most
  Decode8Plan p;
  chunk8_plan(a.C, a.Hq, a.Hkv, a.D, a.n_tiles, a.win_len, &p);
  if (n_tiles < a.n_tiles) {
    p.span = (n_tiles + p.tile_items - 1) / p.tile_items;
    p.tile_items = (n_tiles + p.span - 1) / p.span;
  }
  p.items = p.tile_items + (win_len + D8<64>::WROWS - 1) / D8<64>::WROWS;
  Split8Args s{};
  s.a = Decode8Args{a.q, a.tiles, a.tile_table, nullptr, a.win_k, a.win_v, nullptr, nullptr, nullptr, nullptr, a.out,
                    a.tiles_bytes, a.io, a.win_cap, a.C, a.Hq, a.Hkv, a.G, a.D, a.table_stride, a.format, a.scale, 0,
                    a.err};
  s.pos0 = a.pos0;
  s.n_tiles = n_tiles;
  s.win_start = a.win_start;
  s.win_len = win_len;
  return launch_any<true>(p, s, a.ws, st);
}

}  // namespace kvarn
