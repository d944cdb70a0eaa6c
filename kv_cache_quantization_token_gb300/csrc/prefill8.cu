// prefill8.cu -- causal attention of a chunk of query positions over 8-bit tile records and the
// FP32 window, on tcgen05 tensor cores.
//
//   out[i][h] = sum_j softmax_j(scale q[i][h] . k_j) v_j over keys j with position(j) <= pos0 + i
//
//   image kernel      a CTA per tile and KV head, or per 16 window rows of K or of V: codes, exact in fp16,
//                     or window rows as fp16 pairs hi + lo scaled by a power of two per 16 rows, as operand
//                     images of 64-key blocks, K [key][channel] and V^T [channel][key], in the
//                     128-byte-swizzled K-major layout the tensor cores read, plus the scales.
//   attention kernel  a CTA per KV head, 128 score rows (the G heads of the group x 128 / G positions) and,
//                     when there are few rows, a share of the keys: 8 or 12 softmax warps, two MMA warps and
//                     two copy warps.
//   merge kernel      joins the key shares, when there are several.
// Chunks of few rows run on the decode kernels instead (few_rows() below).
//
// A scale is constant over 16 keys, so it multiplies scores and probabilities and the codes are used as
// they are: S = Q K^T with the query rows scaled by a power of two, then with one reference u per row
//   w = 2^(S kscale c + log2 vscale - u),  O += w V,  l += (sum of w over the 16 keys) / vscale
// so that a weight costs one multiply-add and one exponential. u is the largest weighted score so far,
// moved only when exceeded by several powers of two, so that O is rarely rescaled; whatever the ratio of
// the value scales, the largest terms of O keep their bits.
// Precision: fp32 queries and their weights are pairs hi + lo of fp16 (22 bits), two products per code
// operand. 16-bit queries are exact in one fp16 operand, and then w is rounded to fp16 once (2^-11 of each
// weight at most, an eighth of bf16's rounding of the output, as much as fp16's): one product. That shows in fp16
// outputs: 301 positions of 15 / 3 heads of 64 are 2.5e-4 off the 64-bit result (relative L2) where the output's
// rounding alone is 2.1e-4, and not in bf16 ones (1.67e-3 beside 1.66e-3). With pairs both are at the rounding alone,
// but 25.3 us become 29.4 and 121 at 15,500 tokens 166; adding up the rounded weights instead of w gives 2.3e-4 for
// 8%. So fp32 queries are the way to more bits. Window rows are always pairs. The query and w are read from tensor
// memory (the A operand), so shared memory feeds B operands only; at head_dim 256 the lo part of the query lives in
// shared memory.
//
// What bounds it (512 positions, 32 / 8 heads of 128 over 15,500 tokens, bf16: 121 us, 1,056 TFLOP/s, 56%
// of the measured bf16 rate; images 17 us of it): the softmax warps. A 64-key block costs the tensor pipe 512
// cycles and each of four softmax warps 475 instructions (by counters, the other warps' share in them), of which the
// SM issues 2.6 per cycle. Some 190 are the scores' own (an exponential each, and half a three-way maximum, packed
// multiply-add, packed addition and conversion); the rest (scales and references per 16 keys, hand-overs, moves) has
// not been taken apart. What made it faster, from 207 us: window rows by 16 (their 128-row CTAs were the tail of the
// image grid), softmax groups that take blocks in turn instead of halves of one block, MMA warps that do their waiting beside each
// other's products, hardware barriers for hand-overs, copies of two blocks at a time, one reference instead
// of two. With fp32 (two products of each kind) the tensor pipe bounds it: 183 us against 122 of products.
// Not kept: P in the columns of its scores (S of the next block then waits for PV), one MMA warp, four
// softmax groups (96 registers each), 128-key blocks, one equal stretch of the work per SM (135 us: pipelines
// fill and drain twice, every row block is joined), another order of keys per CTA.
//
// A cached row with a NaN or an infinity gets a NaN key and a zero value in the images: a score row that
// sees it becomes NaN, one that does not is untouched (0 x NaN never enters the value product).
// Every wait is bounded; a CTA that gives up writes NaN rows, frees its TMEM and returns.
#include <math.h>

#include "cache8.cuh"
#include "tcgen05.cuh"

namespace kvarn {
namespace {

constexpr float kHead = 8.f;  // w is about 2^8: lo parts of fp16 pairs stay normal
constexpr float kLag = 7.f;   // references move when exceeded by this power of two
// The tensor core drops what falls below an accumulator's last bit, for fp32 work eight times per block,
// some 1e-8 of O each time: O is emptied into global memory with rounded sums every so many blocks. 36 keep
// fp32 results as close as a plain fp32 computation's (8 heads x 700 positions over 15,400 tokens: 2.2e-6 against
// 2.3e-6; every 48 2.6e-6, never some 8e-6); 15,500 tokens take 183 us, with 48 181, with 24 189.
constexpr int kEmpty = 36;

template <int D, int NP>
struct PC8 {
  static constexpr int KB = 64;                   // image rows of a block: 64 keys of a tile,
  static constexpr int KW = 32;                   // or 32 window keys, hi parts and then lo parts
  static constexpr int SUB = kTile / KB;          // blocks of a tile
  static constexpr int IMG = KB * D * 2;          // bytes of an operand image
  static constexpr int NGB = KB / kGrp;           // scale groups of a block
  // Softmax groups of 4 warps, each with 64 columns of scores. Where tensor memory has room, P has
  // columns of its own, and S of a group's next block is formed while its softmax runs; at head_dim
  // 256 P replaces the scores.
  static constexpr bool SEP = D <= 128;
  static constexpr int NG = D == 256 || (D == 128 && NP == 2) ? 2 : 3;
  static constexpr int PW = SEP ? NP * KB / 2 : 0;  // columns of a group's P
  static constexpr int THREADS = 128 * NG + 128;    // and two MMA warps and two copy warps
  static constexpr bool QL_SMEM = D == 256 && NP == 2;
  static constexpr int R = D <= 128 ? 6 : QL_SMEM ? 2 : 3;  // image slots of the K and of the V ring
  static constexpr int LP = D <= 128 ? 2 : 1;     // blocks of one copy: few waits, where the ring is deep
  static constexpr int QL_BYTES = QL_SMEM ? 128 * D * 2 : 0;
  static constexpr int OFF_K = QL_BYTES;
  static constexpr int OFF_V = OFF_K + R * IMG;
  static constexpr int OFF_BAR = OFF_V + R * IMG;
  static constexpr int OFF_X = OFF_BAR + 256;              // float2 [NG][128]: (u, l) of a row's threads
  static constexpr int OFF_U = OFF_X + NG * 128 * 8;       // float [NG][128]: reference u after a group's block
  static constexpr int OFF_UE = OFF_U + NG * 128 * 4;      // float [128]: reference of the emptied sums
  static constexpr int OFF_MISC = OFF_UE + 128 * 4;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;        // + slack to align the base to 1024
  // tensor memory columns
  static constexpr int T_QH = 0;
  [[maybe_unused]] static constexpr int T_QL = D / 2;
  static constexpr int T_S = D == 256 ? 128 : D / 2 * NP;
  static constexpr int T_P = SEP ? T_S + NG * KB : T_S;    // group g's at T_P + g * (PW or KB)
  static constexpr int PSTEP = SEP ? PW : KB;
  static constexpr int T_O = T_S + NG * (KB + PW);
  static constexpr int TMEM = 512;
  static_assert(kEmpty % NG == 0, "one group empties O");
  static_assert(T_O + D <= TMEM && SMEM <= 227 * 1024, "TMEM and shared memory");
  static_assert(8 * (4 * R + 1) <= 256 && R % LP == 0, "barriers");
};

// Workspace of a call: images [Hkv][pairs of blocks][K, K, V, V], the groups' scales, and the key shares'
// partial results.
struct Plan8 {
  int n_tsub, n_wsub;     // blocks of visible tiles and window rows
  int row_blocks, shares;
  int64_t head_imgs;      // operand images per KV head, two per block
  size_t off_scale, off_ml, off_acc, off_sum, bytes;
};

// Hand-overs between the warps of a CTA go over its hardware barriers (some 20 cycles; a satisfied test
// of an mbarrier costs 60 to 200 beside the tensor core's reads of shared memory). A warp that gave up
// on a copy or a product raises `fail` and still takes part in every hand-over, so that none is left
// waiting; what it computes from then on is discarded.
enum : int { kBarPair = 2, kBarRead = 6, kBarTurn = 6, kBarP = 9, kBarU = 12 };  // + warp % 4, group, MMA warp
template <int THREADS>
__device__ __forceinline__ void hand_over(int id) {
  asm volatile("barrier.cta.arrive.aligned %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void take_over(int id) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

// Place of a block's K image among its head's; the V image is two further.
__host__ __device__ inline int64_t image_index(int sub) { return 4LL * (sub >> 1) + (sub & 1); }

struct Att8Args {
  Prefill8Args a;
  Plan8 p;
  float* scale;  // [Hkv][blocks][8 scales of K, 8 binary logarithms of scales of V]
  float2* ml;    // [shares][C][Hq]
  float* acc;    // [shares][C][Hq][D]
  float4* sum;   // what O is emptied into: [CTA][D / 4][128 rows], one 512-byte line per warp and step
};

// ---------------------------------------------------------------------------
// 32 bytes to an aligned sector.
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&h)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(h[0]), "r"(h[1]), "r"(h[2]),
               "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
               : "memory");
}

// images: of tile blockIdx.x of KV head blockIdx.y, or (past the tiles) of 16 window rows of K or of V
template <int D, int F>
__global__ void __launch_bounds__(256) image8_kernel(const Att8Args s) {
  using P = PC8<D, 1>;
  using R = Rec8<D>;
  constexpr int KB = P::KB, SUB = P::SUB;
  const Prefill8Args& a = s.a;
  const int kvh = blockIdx.y, tid = threadIdx.x;
  const int n_tblk = s.p.n_tsub / SUB;
  pdl_trigger();
  const int n_sub = s.p.n_tsub + s.p.n_wsub;
  uint8_t* head = a.ws + (int64_t)kvh * s.p.head_imgs * P::IMG;
  if ((int)blockIdx.x < n_tblk) {
    const int j = blockIdx.x;
    const int64_t off = a.tile_table[(int64_t)kvh * a.table_stride + j];
    const bool good = !(off & 15) && off >= 0 && off <= a.tiles_bytes - R::kBytes;
    if (!good && tid == 0) report(a.err, KVARN_DEVERR_RECORD);
    const unsigned char* rec = a.tiles + (good ? off : 0);  // (read only if good)
    // 16 D units of 16 codes: K (16 channels of a token), then V (16 tokens of a channel)
    constexpr int UNITS = 16 * D / 256;
    uint4 w[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
      w[i] = good ? *reinterpret_cast<const uint4*>(rec + 16 * (tid + 256 * i)) : make_uint4(0, 0, 0, 0);
    float4 f[4] = {};
    if (good) {
      const float4* sp = reinterpret_cast<const float4*>(rec + R::kKScale);
      f[0] = sp[0]; f[1] = sp[1]; f[2] = sp[2]; f[3] = sp[3];
    }
    const float* fs = &f[0].x;
    unsigned dead = 0;  // groups whose tokens poison what sees them
#pragma unroll
    for (int g = 0; g < kGrps; ++g)
      if (!good || !isfinite(fs[g]) || !isfinite(fs[8 + g])) dead |= 1u << g;
    if (tid < 16) {
      const int g = tid & 7;
      float* sc = s.scale + ((int64_t)kvh * n_sub + (int64_t)j * SUB + g / P::NGB) * 16;
      const float x = (dead >> g & 1) ? 1.f : *reinterpret_cast<const float*>(rec + R::kKScale + 4 * tid);
      sc[(tid >> 3) * 8 + g % P::NGB] = tid < 8 ? x : fast_lg2(x);
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const bool is_v = i >= UNITS / 2;
      const int x = tid + 256 * (is_v ? i - UNITS / 2 : i);
      // unit x: group of 8 rows and run of 64 (blk), row of the group, piece of 16 of the run
      const int piece = x & 3, r8 = (x >> 2) & 7, blk = x >> 5;
      constexpr int RUNS_K = D / 64;
      const int row = (is_v ? blk >> 1 : blk / RUNS_K) * 8 + r8;
      const int k = (is_v ? blk & 1 : blk % RUNS_K) * 64 + piece * 16;
      const int tok = is_v ? k : row;
      uint32_t h[8];
      codes_to_half<F>(w[i].x, h[0], h[1]);
      codes_to_half<F>(w[i].y, h[2], h[3]);
      codes_to_half<F>(w[i].z, h[4], h[5]);
      codes_to_half<F>(w[i].w, h[6], h[7]);
      if (dead >> (tok / kGrp) & 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = is_v ? 0u : 0x7E007E00u;  // 0, or NaN
      }
      uint8_t* img = head + (image_index(j * SUB + tok / KB) + (is_v ? 2 : 0)) * P::IMG;
      const int rr = is_v ? row : row % KB, kk = is_v ? k % KB : k, rows = is_v ? D : KB;
      // the two 16-byte chunks of the unit share a 32-byte sector, swapped in odd rows of the swizzle
      if (rr & 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t t = h[e];
          h[e] = h[4 + e];
          h[4 + e] = t;
        }
      }
      st_sector(img + (sw_off(rr, kk, rows) & ~31u), h);
    }
    return;
  }
  // 16 window rows: pairs hi + lo of row / 2^e, one e for the 16. A block holds 32 window keys: its
  // image's first 32 rows (columns, of V^T) the hi parts, the other 32 the lo parts.
  __shared__ unsigned amax_s;
  __shared__ unsigned bad_s;  // bit t: row t holds a NaN or an infinity
  const int wx = blockIdx.x - n_tblk, g = wx >> 1;
  const bool is_v = wx & 1;
  const int t0 = kGrp * g;  // first window row
  const int sub = s.p.n_tsub + t0 / P::KW, r0 = t0 % P::KW;
  auto row_of = [&](const float* base, int t) {
    return base + ((int64_t)kvh * a.win_cap + (a.win_start + t0 + t) % a.win_cap) * D;
  };
  if (tid == 0) amax_s = bad_s = 0u;
  __syncthreads();
  // one pass over the rows of this tensor for the largest magnitude, over both for bad rows
  unsigned m = 0u;
  for (int u = tid; u < 2 * kGrp * D / 4; u += 256) {
    const bool v2 = u >= kGrp * D / 4;
    const int x = v2 ? u - kGrp * D / 4 : u, t = x / (D / 4);
    if (t0 + t < a.win_len) {
      const uint4 y = *reinterpret_cast<const uint4*>(row_of(v2 ? a.win_v : a.win_k, t) + 4 * (x % (D / 4)));
      const unsigned z = max(max(y.x & 0x7FFFFFFFu, y.y & 0x7FFFFFFFu), max(y.z & 0x7FFFFFFFu, y.w & 0x7FFFFFFFu));
      if (z >= 0x7F800000u) atomicOr(&bad_s, 1u << t);
      else if (v2 == is_v) m = max(m, z);
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) atomicMax(&amax_s, m);
  __syncthreads();
  const float f = pow2_to(__uint_as_float(amax_s), 8);
  const unsigned bad = bad_s;
  if (tid < 2)  // (the lo rows have their hi rows' scale)
    s.scale[((int64_t)kvh * n_sub + sub) * 16 + (is_v ? 8 : 0) + r0 / kGrp + 2 * tid] =
        is_v ? fast_lg2(pow2_inverse(f)) : pow2_inverse(f);
  uint8_t* img = head + (image_index(sub) + (is_v ? 2 : 0)) * P::IMG;
  for (int u = tid; u < 2 * D; u += 256) {  // 8 elements along the summed index: channels of K, tokens of V
    const int row = is_v ? u % D : u / (D / 8), k = is_v ? (u / D) * 8 : (u % (D / 8)) * 8;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = is_v ? k + i : row;
      v[i] = 0.f;
      if (t0 + t < a.win_len) {
        const float x = is_v ? row_of(a.win_v, t)[row] : row_of(a.win_k, t)[k + i];
        v[i] = (bad >> t & 1) ? (is_v ? 0.f : NAN) : f * x;
      }
    }
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_pair(v[2 * i], v[2 * i + 1], h[i], l[i]);
    const uint32_t oh = is_v ? sw_off(row, r0 + k, D) : sw_off(r0 + row, k, KB);
    const uint32_t ol = is_v ? sw_off(row, P::KW + r0 + k, D) : sw_off(P::KW + r0 + row, k, KB);
    *reinterpret_cast<uint4*>(img + oh) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(img + ol) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// ---------------------------------------------------------------------------
template <int D, int NP>
__global__ void __launch_bounds__(PC8<D, NP>::THREADS, 1) attend8_kernel(const Att8Args s) {
  using P = PC8<D, NP>;
  constexpr int KB = P::KB, KW = P::KW, R = P::R, NGB = P::NGB, NG = P::NG;
  const Prefill8Args& a = s.a;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~uintptr_t(1023));
  uint64_t* bar_fk = reinterpret_cast<uint64_t*>(sm + P::OFF_BAR);  // [R] K image landed
  uint64_t* bar_dk = bar_fk + R;    // [R] S of its block complete
  uint64_t* bar_fv = bar_dk + R;    // [R] V image landed
  uint64_t* bar_dv = bar_fv + R;    // [R] PV of its block complete
  uint64_t* bar_o = bar_dv + R;     // every product complete (one arrival per MMA warp)
  float2* xm = reinterpret_cast<float2*>(sm + P::OFF_X);
  float* su = reinterpret_cast<float*>(sm + P::OFF_U);
  [[maybe_unused]] float* su_empty = reinterpret_cast<float*>(sm + P::OFF_UE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + P::OFF_MISC);
  volatile int* fail = reinterpret_cast<volatile int*>(sm + P::OFF_MISC + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = tid & 127, half = (tid >> 7) & 1;
  const int kvh = blockIdx.y, share = blockIdx.z;
  const int ppc = 128 / a.G, i0 = blockIdx.x * ppc;
  const int my_g = row / ppc, my_i = i0 + row % ppc;
  const bool my_valid = my_i < a.C && my_g < a.G;
  const int64_t my_pos = a.pos0 + my_i;
  const int64_t pmin = a.pos0 + i0, pmax = a.pos0 + min(a.C, i0 + ppc) - 1;
  const int hq = kvh * a.G + min(my_g, a.G - 1);
  const int64_t out_row = ((int64_t)share * a.C + my_i) * a.Hq + hq;  // among the key shares' results
  [[maybe_unused]] float4* sums =
      s.sum + (((int64_t)share * gridDim.y + kvh) * gridDim.x + blockIdx.x) * (D / 4) * 128;
  const int64_t win_pos0 = 128LL * a.n_tiles;
  // blocks this CTA sees: tiles up to pmax, window blocks up to pmax; its share of them
  const int n_sub = s.p.n_tsub + s.p.n_wsub;
  int vis_t = (int)min((int64_t)s.p.n_tsub, pmax / KB + 1);
  int vis_w = pmax >= win_pos0 ? (int)min((int64_t)s.p.n_wsub, (pmax - win_pos0) / KW + 1) : 0;
  const int vis = vis_t + vis_w;
  const int pairs = (vis + 1) / 2;  // shares are whole pairs of blocks
  const int b0 = 2 * (int)((int64_t)pairs * share / s.p.shares);
  const int b1 = min(vis, 2 * (int)((int64_t)pairs * (share + 1) / s.p.shares));
  const int n_blk = b1 - b0;
  auto sub_of = [&](int j) { const int v = b0 + j; return v < vis_t ? v : s.p.n_tsub + (v - vis_t); };
  const uint8_t* head = a.ws + (int64_t)kvh * s.p.head_imgs * P::IMG;

  if (tid == 0) {
    for (int i = 0; i < 4 * R; ++i) mbar_init_n(bar_fk + i, 1);
    mbar_init_n(bar_o, 2);
    mbar_fence_init();
    *fail = 0;
  }
  if (warp == 0) tmem_alloc(tmem_slot, P::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem + P::T_O;
  const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;

  // copies, by one thread for the K images and one for the V images; the first fill of the rings is requested
  // before the queries are prepared
  const bool copies = warp >= 4 * NG + 2 && lane == 0, is_v = warp == 4 * NG + 3;
  uint64_t* full = is_v ? bar_fv : bar_fk;
  auto copy = [&](int t) {  // of blocks t .. t + LP - 1 (a pair's second image is copied even if no row sees it)
    const int sl = t % R;
    mbar_arrive_tx(full + sl, P::LP * P::IMG);
    bulk_in(sm + (is_v ? P::OFF_V : P::OFF_K) + sl * P::IMG,
            head + (image_index(sub_of(t)) + (is_v ? 2 : 0)) * P::IMG, P::LP * P::IMG, full + sl);
  };
  if (copies) {
    pdl_wait();  // the images of this call are complete
    for (int t = 0; t < min(n_blk, R); t += P::LP) copy(t);
  }

  // query rows into TMEM: scaled by a power of two, fp16 (hi and lo); two threads per row
  if (tid < 256) {
    const int64_t at = ((int64_t)my_i * a.Hq + hq) * D + half * (D / 2);
    float m = 0.f;
    if (my_valid)
#pragma unroll 8
      for (int c = 0; c < D / 2; c += 4) {
        const float4 v = io_ld4(a.q, a.io, at + c);
        m = fmaxf(fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
      }
    xm[half * 128 + row].x = m;
    take_over<64>(kBarPair + (warp & 3));
    const float mq = fmaxf(m, xm[(half ^ 1) * 128 + row].x), up = pow2_to(mq, 10);
    if (half == 0) xm[row].y = fabsf(a.scale) * pow2_inverse(up);
    // (maxima are taken before the positive scales; a row with an infinity becomes NaN)
    const float p2 = mq == INFINITY ? NAN : copysignf(up, a.scale);
#pragma unroll 1
    for (int c0 = 0; c0 < D / 2; c0 += 32) {
      uint32_t hw[16], lw[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 v = my_valid ? io_ld4(a.q, a.io, at + c0 + 4 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
        split_pair(v.x * p2, v.y * p2, hw[2 * e], lw[2 * e]);
        split_pair(v.z * p2, v.w * p2, hw[2 * e + 1], lw[2 * e + 1]);
      }
      tmem_st16(tmem + lb + P::T_QH + half * (D / 4) + c0 / 2, hw);
      if constexpr (NP == 2 && !P::QL_SMEM) tmem_st16(tmem + lb + P::T_QL + half * (D / 4) + c0 / 2, lw);
      if constexpr (P::QL_SMEM) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(sm + sw_off(row, half * (D / 2) + c0 + 8 * e, 128)) =
              make_uint4(lw[4 * e], lw[4 * e + 1], lw[4 * e + 2], lw[4 * e + 3]);
      }
    }
    tmem_wait_st();
    if constexpr (P::QL_SMEM) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const float qscale = xm[row].y;  // what turns a product into a score, but for the key's scale
  float u_own = -INFINITY, l_part = 0.f;  // softmax threads: sum of probabilities, in units of 2^u_own
  if (warp >= 4 * NG + 2) {
    // ---------------- the copies that follow
    if (copies) {
      uint64_t* done = is_v ? bar_dv : bar_dk;
      int t = min((n_blk + P::LP - 1) / P::LP * P::LP, R);
      for (; t < n_blk; t += P::LP) {
        const int last = t - R + P::LP - 1;  // the last block that used the slots
        mbar_wait8(done + last % R, (uint32_t)(last / R) & 1u, a.err, fail);
        copy(t);
      }
      // every copy has landed before the CTA can retire
      for (int i = max(0, t - R); i < t; i += P::LP)
        mbar_wait8(full + i % R, (uint32_t)(i / R) & 1u, a.err);
    }
    __syncwarp();
  } else if (warp >= 4 * NG) {
    // ---------------- products, by two warps: each waits for its operands while the tensor pipe works on
    // what the other issued (a satisfied wait costs some 200 cycles beside the softmax warps, more than the
    // pipe's short queue lasts). The whole warp runs the loop, so that operand addresses stay uniform, and
    // one elected lane issues; the loops are unrolled over the rings, so that slots, addresses and
    // descriptors are constants.
    if (n_blk > 0) {
      const uint64_t dk = sdesc(smem_addr(sm + P::OFF_K)), dv = sdesc(smem_addr(sm + P::OFF_V));
      [[maybe_unused]] const uint64_t dq = sdesc(smem_addr(sm));  // lo part of the query (head_dim 256)
      constexpr uint32_t kStep = P::IMG >> 4;
      auto wait = [&](uint64_t* bar, uint32_t par) { mbar_wait8(bar, par, a.err, fail); };
      // S of a block from the K image in slot sl into columns ss
      auto s_products = [&](int sl, int ss) {
        const uint64_t kd = dk + sl * kStep;
        const uint32_t t_s = tmem + P::T_S + KB * ss;
#pragma unroll
        for (int h = NP - 1; h >= 0; --h) {  // the query's lo part first: while the sums are small
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t bd = sdesc_add(kd, (kk >> 2) * KB * 128 + (kk & 3) * 32);
            const uint32_t acc = h < NP - 1 || kk > 0;
            if (P::QL_SMEM && h == 1)
              mma_ss(t_s, sdesc_add(dq, (kk >> 2) * 128 * 128 + (kk & 3) * 32), bd, idesc_f16<KB>(), acc);
            else
              mma_ts(t_s, tmem + (h == 1 ? P::T_QL : P::T_QH) + 8 * kk, bd, idesc_f16<KB>(), acc);
          }
        }
        mma_commit(bar_dk + sl);
      };
      // O += P V: the V image in slot sl, P in columns ss (32 columns hi, then 32 lo)
      auto o_products = [&](int sl, int ss, bool first) {
        const uint64_t vd = dv + sl * kStep;
        const uint32_t t_p = tmem + P::T_P + P::PSTEP * ss;
#pragma unroll
        for (int kk = 0; kk < KB / 16; ++kk) {
          const uint64_t bd = sdesc_add(vd, kk * 32);
          mma_ts(t_o, t_p + 8 * kk, bd, idesc_f16<D>(), !first || kk > 0);
          if (NP == 2) mma_ts(t_o, t_p + 32 + 8 * kk, bd, idesc_f16<D>(), 1);
        }
        mma_commit(bar_dv + sl);
      };
      constexpr int U0 = (R % NG == 0) ? R : R * NG;
      if constexpr (!P::SEP) {
        // the pipe's order alone keeps S(t) behind PV(t - NG), whose P is in the same columns: the warps take
        // turns at steps of the two, handing over once a step is issued
        constexpr int U = U0 % 2 == 0 ? U0 : 2 * U0;
        const int me = warp - 4 * NG, n_steps = n_blk + NG;
        for (int t0 = 0; t0 < n_steps; t0 += U) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int t = t0 + u;
            if (t >= n_steps) break;
            if ((u & 1) != me) continue;
            const int sl = u % R, ss = u % NG, sv = (u + R * NG - NG) % R;
            if (t >= NG) wait(bar_fv + sv, (uint32_t)((t - NG) / R) & 1u);
            if (t < n_blk && R > 2) wait(bar_fk + sl, (uint32_t)(t / R) & 1u);
            __syncwarp();
            if (t >= NG) take_over<160>(kBarP + ss);
            if (t > 0) take_over<64>(kBarTurn + me);
            tc_fence_after();
            if (t >= NG && elect_one()) o_products(sv, ss, NP == 2 ? (t - NG) % kEmpty == 0 : t == NG);
            __syncwarp();
            if (t < n_blk && R == 2) {  // (a ring of two: its K image is as late as this)
              wait(bar_fk + sl, (uint32_t)(t / R) & 1u);
              __syncwarp();
              tc_fence_after();
            }
            if (t < n_blk && elect_one()) s_products(sl, ss);
            __syncwarp();
            tc_fence_before();
            if (t + 1 < n_steps) hand_over<64>(kBarTurn + (me ^ 1));
          }
        }
      } else if (warp == 4 * NG) {  // S, into columns whose scores have been read
        for (int t0 = 0; t0 < n_blk; t0 += U0) {
#pragma unroll
          for (int u = 0; u < U0; ++u) {
            const int t = t0 + u;
            if (t >= n_blk) break;
            const int sl = u % R, ss = u % NG;
            if (u % P::LP == 0) wait(bar_fk + sl, (uint32_t)(t / R) & 1u);
            __syncwarp();
            if (t >= NG) take_over<160>(kBarRead + ss);
            tc_fence_after();
            if (elect_one()) s_products(sl, ss);
            __syncwarp();
          }
        }
      } else {  // PV
        for (int t0 = 0; t0 < n_blk; t0 += U0) {
#pragma unroll
          for (int u = 0; u < U0; ++u) {
            const int t = t0 + u;
            if (t >= n_blk) break;
            const int sl = u % R, ss = u % NG;
            if (u % P::LP == 0) wait(bar_fv + sl, (uint32_t)(t / R) & 1u);
            __syncwarp();
            take_over<160>(kBarP + ss);
            tc_fence_after();
            if (elect_one()) o_products(sl, ss, NP == 2 ? t % kEmpty == 0 : t == 0);
            __syncwarp();
          }
        }
      }
      // everything issued has completed before the CTA goes on: a commit behind it all
      if (elect_one()) mma_commit(bar_o);
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait8(bar_o, 0, a.err))) *fail = 1;
    }
    __syncwarp();
  } else {
    // ---------------- softmax: one thread per row; the groups of four warps take the blocks in turn,
    // so that the latencies of one are covered by the others' arithmetic. m and l are a thread's own;
    // u, which scales O, is decided block after block and handed from group to group.
    const int grp = warp >> 2, grp_before = (grp + NG - 1) % NG;
    const uint32_t t_s = tmem + P::T_S + KB * grp + lb, t_p = tmem + P::T_P + P::PSTEP * grp + lb;
    // a block's scales are read from L2 while the group's block before it is worked on
    const int n_t = max(0, min(n_blk, vis_t - b0));  // tile blocks; window blocks follow
    // of them, the leading ones that every row of the CTA sees whole
    const int n_full = (int)max((int64_t)0, min((int64_t)n_t, (pmin + 1) / KB - b0));
    const float* scales = s.scale + (int64_t)kvh * n_sub * 16;
    float ks_next[NGB] = {}, lv_next[NGB] = {};
    auto fetch_scales = [&](int j) {
      const float4* p = reinterpret_cast<const float4*>(scales + 16 * (j < n_t ? b0 + j : sub_of(j)));
#pragma unroll
      for (int g = 0; g < NGB; g += 4) {
        const float4 x = p[g / 4], y = p[2 + g / 4];
        ks_next[g] = x.x; ks_next[g + 1] = x.y; ks_next[g + 2] = x.z; ks_next[g + 3] = x.w;
        lv_next[g] = y.x; lv_next[g + 1] = y.y; lv_next[g + 2] = y.z; lv_next[g + 3] = y.w;
      }
    };
    pdl_wait();  // the scales belong to this call's images
    if (grp < n_blk) fetch_scales(grp);
    auto wait = [&](uint64_t* bar, uint32_t par) { mbar_wait8(bar, par, a.err, fail); };
    int sl = grp, sl_before = 0;  // ring slot of block j and of the group's block before, and their parities
    uint32_t ph = 0, ph_before = 0;
    for (int j = grp; j < n_blk; j += NG) {
      float ks[NGB], lv[NGB];
#pragma unroll
      for (int g = 0; g < NGB; ++g) {
        // (not zero, so that a hidden key's -inf stays; a factor that small makes every score 0 anyway)
        ks[g] = fmaxf(ks_next[g] * qscale, 1e-37f);
        lv[g] = lv_next[g];
      }
      if (j + NG < n_blk) fetch_scales(j + NG);
      wait(bar_dk + sl, ph);
      __syncwarp();
      tc_fence_after();
      float sv[KB];
      tmem_ld32_nowait(t_s, *reinterpret_cast<uint32_t(*)[32]>(sv));
      tmem_ld32_nowait(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32));
      // P's columns are free when the product that read the group's block before is complete
      const bool p_free = !P::SEP || j < NG || mbar_done(bar_dv + sl_before, ph_before);
      tmem_wait_ld(sv);
      if (P::SEP) {
        tc_fence_before();
        if (j + NG < n_blk) hand_over<160>(kBarRead + grp);
      }
      if (j >= n_full) {  // keys of the block that this row sees
        const int sub = sub_of(j);
        const bool is_tile = sub < s.p.n_tsub;
        const int64_t kpos0 = is_tile ? (int64_t)KB * sub : win_pos0 + (int64_t)KW * (sub - s.p.n_tsub);
        const int nkeys = is_tile ? KB : min(KW, a.win_len - KW * (sub - s.p.n_tsub));
        if (!is_tile) {
#pragma unroll
          for (int u = 0; u < KW; ++u) sv[u] += sv[KW + u];  // hi and lo part of a key
        }
        const int seen = !my_valid ? 0 : (int)max((int64_t)0, min((int64_t)nkeys, my_pos - kpos0 + 1));
#pragma unroll
        for (int u = 0; u < KB; ++u)
          if (u >= seen) sv[u] = -INFINITY;
      }
      // largest score of each group of keys, and of the row's weighted scores
      float mg[NGB], ublk = -INFINITY;
#pragma unroll
      for (int g = 0; g < NGB; ++g) {
        float m = sv[16 * g];
#pragma unroll
        for (int u = 1; u < 15; u += 2) m = fmax3(m, sv[16 * g + u], sv[16 * g + u + 1]);
        mg[g] = fmaxf(m, sv[16 * g + 15]) * ks[g];
        ublk = fmaxf(ublk, mg[g] + lv[g]);
      }
      // u after the block before, from the group that has it
      float u_old = -INFINITY;
      if (j > 0) {
        take_over<256>(kBarU + grp_before);
        u_old = su[grp_before * 128 + row];
      }
      const bool need = ublk > u_old + kLag;
      const float u_ref = need ? ublk : u_old;
      su[grp * 128 + row] = u_ref;
      if (j + 1 < n_blk) hand_over<256>(kBarU + grp);
      // (a row with no visible key yet has scores of -inf only, and any reference does)
      const float u = u_ref == -INFINITY ? 0.f : u_ref;
      l_part *= u_own != -INFINITY ? fast_ex2(u_own - u_ref) : 1.f;
      u_own = u_ref;
      uint32_t hw[KB / 2], lw[KB / 2];
#pragma unroll
      for (int g = 0; g < NGB; ++g) {
        // a group whose weights vanish beside the row's largest (2^-kHead of a step of fp16) is given more
        // weight, none of which reaches the product, so that l still counts its probabilities
        const float le = fmaxf(lv[g], u - fmaxf(mg[g], -1e30f) - (kHead + 50.f));
        const float2 k2 = make_float2(ks[g], ks[g]), c2 = make_float2(le + kHead - u, le + kHead - u);
        float2 ls2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = __ffma2_rn(make_float2(sv[16 * g + 2 * e], sv[16 * g + 2 * e + 1]), k2, c2);
          const float2 w = make_float2(fast_ex2(x.x), fast_ex2(x.y));
          ls2 = __fadd2_rn(ls2, w);
          if constexpr (NP == 2) {
            split_pair(w.x, w.y, hw[8 * g + e], lw[8 * g + e]);
          } else {
            const __half2 h = __floats2half2_rn(w.x, w.y);
            hw[8 * g + e] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        l_part = fmaf(ls2.x + ls2.y, fast_ex2(-le - kHead), l_part);
      }
      if (j >= n_t) {  // a window key's weight meets both parts of its value
#pragma unroll
        for (int e = 0; e < KW / 2; ++e) {
          hw[KW / 2 + e] = hw[e];
          if constexpr (NP == 2) lw[KW / 2 + e] = lw[e];
        }
      }
      if (!p_free) wait(bar_dv + sl_before, ph_before);
      __syncwarp();
      if (P::SEP) tc_fence_after();
      sl_before = sl;
      ph_before = ph;
      sl += NG;
      if (sl >= R) {
        sl -= R;
        ph ^= 1u;
      }
      // w: hi in 32 columns, lo in the 32 after
      tmem_st32_nowait(t_p, hw);
      if constexpr (NP == 2) tmem_st32_nowait(t_p + 32, lw);
      // O belongs to the previous block's product until that completes
      if (NP == 2 && j > 0 && j % kEmpty == 0) {
        wait(bar_dv + (j - 1) % R, (uint32_t)((j - 1) / R) & 1u);
        __syncwarp();
        tc_fence_after();
        const float u_sum = su_empty[row], again = j > kEmpty && u_sum != -INFINITY ? fast_ex2(u_sum - u_old) : 0.f;
        float4* dst = sums + row;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float v[32];
          float4 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            y[i] = again != 0.f ? __ldcg(dst + (c0 / 4 + i) * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
          tmem_ld32(t_o + lb + c0, v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(dst + (c0 / 4 + i) * 128,
                   make_float4(fmaf(y[i].x, again, v[4 * i]), fmaf(y[i].y, again, v[4 * i + 1]),
                               fmaf(y[i].z, again, v[4 * i + 2]), fmaf(y[i].w, again, v[4 * i + 3])));
        }
        su_empty[row] = u_old;
      } else if (j > 0 && __any_sync(0xffffffffu, need)) {
        const float alpha = need && u_old != -INFINITY ? fast_ex2(u_old - u_ref) : 1.f;
        wait(bar_dv + (j - 1) % R, (uint32_t)((j - 1) / R) & 1u);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float v[32];
          tmem_ld32(t_o + lb + c0, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= alpha;
          tmem_st32(t_o + lb + c0, v);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      hand_over<160>(kBarP + grp);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool ok = *fail == 0;
  if (warp < 4 * NG) xm[(warp >> 2) * 128 + row] = make_float2(u_own, l_part);
  __syncthreads();
  // ---- epilogue: half of a row's channels per thread
  if (tid < 256) {
    // O and the sum l in units of 2^u, u after the last block
    const float u = n_blk > 0 ? su[((n_blk - 1) % NG) * 128 + row] : -INFINITY;
    float l = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float2 v = xm[g * 128 + row];
      l += v.x != -INFINITY ? v.y * fast_ex2(v.x - u) : v.y;  // (no reference: 0, or NaN of NaN scores)
    }
    float f = pow2_inverse(256.f);  // 2^-kHead
    if (s.p.shares == 1) f = l != 0.f ? f / l : 0.f;
    if (!ok) f = NAN;
    const int64_t orow = (int64_t)my_i * a.Hq + hq;
    // what O was emptied of, in units of 2^su_empty
    const bool emptied = NP == 2 && n_blk > kEmpty;
    const float u_sum = emptied ? su_empty[row] : -INFINITY;
    const float again = u_sum != -INFINITY ? fast_ex2(u_sum - u) : 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < D / 2; c0 += 32) {
      float v[32];
      if (n_blk > 0 && ok) {
        tmem_ld32(t_o + lb + half * (D / 2) + c0, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
      }
      if (my_valid) {
        if (again != 0.f) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 y = __ldcg(sums + (half * (D / 8) + (c0 + i) / 4) * 128 + row);
            v[i] = fmaf(y.x, again, v[i]); v[i + 1] = fmaf(y.y, again, v[i + 1]);
            v[i + 2] = fmaf(y.z, again, v[i + 2]); v[i + 3] = fmaf(y.w, again, v[i + 3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 o = make_float4(v[i] * f, v[i + 1] * f, v[i + 2] * f, v[i + 3] * f);
          const int c = half * (D / 2) + c0 + i;
          if (s.p.shares == 1) io_st4(a.out, a.io, orow * D + c, o);
          else *reinterpret_cast<float4*>(s.acc + out_row * D + c) = o;
        }
      }
    }
    if (s.p.shares > 1 && my_valid && half == 0)
      s.ml[out_row] = ok ? make_float2(u, l) : make_float2(0.f, NAN);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, P::TMEM);
}

// ---------------------------------------------------------------------------
// sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s for each (position, head); D / 4 threads per row
template <int D>
__global__ void __launch_bounds__(256) join8_kernel(const Att8Args s) {
  pdl_wait();
  const Prefill8Args& a = s.a;
  const int64_t rows = (int64_t)a.C * a.Hq;
  const int64_t r = (int64_t)blockIdx.x * (1024 / D) + threadIdx.x / (D / 4);
  const int c = 4 * (threadIdx.x % (D / 4));
  if (r >= rows) return;
  float M = -INFINITY;
  for (int i = 0; i < s.p.shares; ++i) M = fmaxf(M, s.ml[i * rows + r].x);
  float L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < s.p.shares; ++i) {
    const float2 ml = s.ml[i * rows + r];
    if (ml.y == 0.f) continue;
    const float w = fast_ex2(ml.x - M);
    const float4 v = *reinterpret_cast<const float4*>(s.acc + (i * rows + r) * D + c);
    L = fmaf(w, ml.y, L);
    o.x = fmaf(w, v.x, o.x); o.y = fmaf(w, v.y, o.y); o.z = fmaf(w, v.z, o.z); o.w = fmaf(w, v.w, o.w);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  io_st4(a.out, a.io, r * D + c, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

Plan8 plan8(int C, int n_tblk, int win_vis, int Hq, int Hkv, int D, bool fp32) {
  Plan8 p;
  const int KB = PC8<64, 1>::KB, G = Hq / Hkv, ppc = 128 / G;
  p.n_tsub = n_tblk * (kTile / KB);
  p.n_wsub = (win_vis + 2 * PC8<64, 1>::KW - 1) / (2 * PC8<64, 1>::KW) * 2;
  p.head_imgs = 2LL * (p.n_tsub + p.n_wsub);
  p.row_blocks = (int)(((int64_t)C + ppc - 1) / ppc);
  const int64_t ctas = (int64_t)p.row_blocks * Hkv;
  int64_t shares = ctas > 0 ? sm_count() / ctas : 1;
  const int64_t most = (p.n_tsub + p.n_wsub) / 4;  // two pairs of blocks per share at least
  if (shares > most) shares = most;
  if (shares > 64) shares = 64;
  p.shares = shares < 1 ? 1 : (int)shares;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p.off_scale = up((size_t)Hkv * p.head_imgs * KB * D * 2);
  p.off_ml = p.off_scale + up((size_t)Hkv * (p.n_tsub + p.n_wsub) * 64);
  const size_t rows = p.shares > 1 ? (size_t)p.shares * C * Hq : 0;
  p.off_acc = p.off_ml + up(rows * sizeof(float2));
  p.off_sum = p.off_acc + up(rows * D * sizeof(float));
  const bool emptied = fp32 && p.n_tsub + p.n_wsub > kEmpty;
  p.bytes = p.off_sum + (emptied ? up((size_t)ctas * p.shares * 128 * D * sizeof(float)) : 0);
  return p;
}

template <int D, int F, int NP>
cudaError_t launch_p8(const Att8Args& s, cudaStream_t st) {
  using P = PC8<D, NP>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(attend8_kernel<D, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int blocks = s.p.n_tsub / P::SUB + 2 * s.p.n_wsub * (P::KW / kGrp);
  image8_kernel<D, F><<<dim3(blocks, s.a.Hkv), 256, 0, st>>>(s);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  LaunchCfg L(dim3(s.p.row_blocks, s.a.Hkv, s.p.shares), dim3(P::THREADS), P::SMEM, st, KVARN_LAUNCH_PDL);
  e = cudaLaunchKernelEx(&L.cfg, attend8_kernel<D, NP>, s);
  if (e != cudaSuccess || s.p.shares == 1) return e;
  const int64_t rows = (int64_t)s.a.C * s.a.Hq;
  LaunchCfg J(dim3((unsigned)((rows + 1024 / D - 1) / (1024 / D))), dim3(256), 0, st, KVARN_LAUNCH_PDL);
  return cudaLaunchKernelEx(&J.cfg, join8_kernel<D>, s);
}

template <int D>
cudaError_t launch_p8d(const Att8Args& s, cudaStream_t st) {
  const bool e = s.a.format == KVARN_CODE8_E4M3;
  if (s.a.io == KVARN_IO_F32) return e ? launch_p8<D, 1, 2>(s, st) : launch_p8<D, 0, 2>(s, st);
  return e ? launch_p8<D, 1, 1>(s, st) : launch_p8<D, 0, 1>(s, st);
}

// Chunks of few score rows per KV head go to the decode kernels, which need no images but go over the cache once
// for every eight rows ("group"). Per tile-head they take some 5 ns a group (head_dim 64: 3, 256: 8) and per 128 window rows
// 10 times that, fp32 rows through tf32 products; the images with their kernels take 5 tiles' worth of a group
// per tile, 4 groups' worth per window row, and some 5 us more, and with fewer than 6 KV heads no less than with 6.
// At head_dim 128, 8 KV heads, bf16 (us, decode kernels against images): 8 groups over 40 tiles 23.4 / 26.0, 12
// 34.4 / 28.1; 5 over 128 tiles 36.3 / 38.1, 6 42.2 / 39.3; no tiles and 1,000 window rows, 4 groups 19.1 / 21.5, 6
// 26.3 / 22.6, 64 221 / 29; 2 KV heads, 16 groups over 128 tiles 30.1 / 48.9, 24 42.1 / 38.4; head_dim 64, 8 over 15
// tiles 11.3 / 13.7, 24 24.2 / 16.2; head_dim 256, 8 over 40 tiles 34.2 / 39.0, 12 50.3 / 43.6. Over 800 sizes (1 to 8 KV
// heads, 4 to 64 groups, 0 to 128 tiles, 60 to 3,000 window rows) the choice costs 0.4% on the mean, 31% at worst.
constexpr int64_t kFewGroups = 64, kFewWork = 1600;
int64_t row_groups(int C, int G) { return ((int64_t)C * G + 7) / 8; }
int64_t few_heads(int Hkv) { return Hkv > 6 ? Hkv : 6; }
bool few_rows(int C, int G, int Hkv, int n_tiles, int win_len) {
  const int64_t groups = row_groups(C, G), work = groups * Hkv, heads = few_heads(Hkv);
  return groups <= kFewGroups &&
         12 * (work - 5 * heads) * n_tiles + (work - 4 * heads) * win_len <= 12 * kFewWork;
}

}  // namespace

size_t prefill8_ws_bytes(int C, int n_tiles, int win_len, int Hq, int Hkv, int D) {
  if (few_rows(C, Hq / Hkv, Hkv, n_tiles, win_len)) {
    Decode8Plan p;
    chunk8_plan(C, Hq, Hkv, D, n_tiles, win_len, &p);
    return p.ws_bytes;
  }
  // shares (and with them the partial results) grow as the visible blocks do
  return plan8(C, n_tiles, win_len, Hq, Hkv, D, true).bytes;
}

// At least prefill8_ws_bytes of every call of at most C positions, n_tiles tiles and win_len window rows, whichever
// kernels serve it: a workspace for a prompt's last chunk is one for all before it.
size_t prefill8_ws_bound(int C, int n_tiles, int win_len, int Hq, int Hkv, int D) {
  const int64_t n = n_tiles, w = win_len, heads = few_heads(Hkv), sms = sm_count();
  const int64_t groups = row_groups(C, Hq / Hkv), work = (groups < kFewGroups ? groups : kFewGroups) * Hkv;
  auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  // Decode kernels: 8 work' rows of tile_items + ceil(w' / 64) entries for a call's own work' <= work. tile_items is at
  // most n' / 16 + slots / work' + 1 (make_plan), and where few_rows holds work' n' <= kFewWork + 5 heads n' and
  // work' w' <= 12 kFewWork + 5 heads w'.
  const int64_t slots = 4 * sms;  // resident CTAs, at most four per SM
  const int64_t entries = 8 * (least(work * n, kFewWork + 5 * heads * n) / 16 + 1 +
                               least(work * w, 12 * kFewWork + 5 * heads * w) / 64 + 1 + 2 * work + slots);
  const size_t few = up((size_t)entries * sizeof(float2)) + up((size_t)entries * D * sizeof(float));
  if (groups * Hkv <= 4 * heads) return few;  // (few_rows holds for every smaller call)
  // Images: those of this call, and the results of key shares, of which there are only as many as fill the SMs
  // once (128 rows to a CTA), and O's emptied sums, of a CTA's rows each.
  const Plan8 p = plan8(C, n_tiles, win_len, Hq, Hkv, D, true);
  const int64_t ctas = (int64_t)p.row_blocks * Hkv;
  const size_t rows = 128 * (size_t)sms, sums = 128 * (size_t)(ctas > sms ? ctas : sms);
  const size_t images = p.off_ml + up(rows * sizeof(float2)) + up(rows * D * sizeof(float)) + up(sums * D * sizeof(float));
  return few > images ? few : images;
}

cudaError_t launch_prefill8(const Prefill8Args& a, cudaStream_t st) {
  // tiles and window rows that the chunk's last position sees: neither path reads others
  const int64_t pmax = a.pos0 + a.C - 1;
  const int n_tblk = (int)(pmax / kTile + 1 < a.n_tiles ? pmax / kTile + 1 : a.n_tiles);
  const int64_t w = pmax - 128LL * a.n_tiles + 1;
  const int win_vis = (int)(w < 0 ? 0 : w < a.win_len ? w : a.win_len);
  // (the path follows from what the workspace was counted for, which does not know the position)
  if (few_rows(a.C, a.G, a.Hkv, a.n_tiles, a.win_len)) return launch_chunk8(a, n_tblk, win_vis, st);
  Att8Args s;
  s.a = a;
  s.p = plan8(a.C, n_tblk, win_vis, a.Hq, a.Hkv, a.D, a.io == KVARN_IO_F32);
  s.scale = reinterpret_cast<float*>(a.ws + s.p.off_scale);
  s.ml = reinterpret_cast<float2*>(a.ws + s.p.off_ml);
  s.acc = reinterpret_cast<float*>(a.ws + s.p.off_acc);
  s.sum = reinterpret_cast<float4*>(a.ws + s.p.off_sum);
  switch (a.D) {
    case 64: return launch_p8d<64>(s, st);
    case 128: return launch_p8d<128>(s, st);
    case 256: return launch_p8d<256>(s, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvarn
