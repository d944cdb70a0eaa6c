// attend.cuh -- causal attention of a chunk of query positions over operand images of a cache, on
// tcgen05 tensor cores: the kernels behind chunked prefill over the 8-bit and the 4-bit cache.
//
//   attention kernel  a CTA per KV head, 128 score rows (the G heads of the group x 128 / G positions) and,
//                     when there are few rows, a share of the keys: 8 or 12 softmax warps, two MMA warps and
//                     two copy warps.
//   join kernel       joins the key shares, when there are several.
//
// The images hold 64-key blocks, K [key][channel] and V^T [channel][key], in the 128-byte-swizzled K-major layout
// the tensor cores read. With SC the keys and values of 16 keys at a time have scales, which multiply scores and
// probabilities, and window rows may follow the tiles; without it the images hold the values themselves, and there
// is no window.
#pragma once

#include <math.h>

#include <type_traits>

#include "cache4.cuh"
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

// ---------------------------------------------------------------------------
// NP: parts of queries and weights, 2 for fp32 calls and 1 for those of 16-bit types. (One fp16 number for a weight: 2^-11 of it
// at most, where half a step of a bf16 output is 2^-9 and of an fp16 output 2^-12 to 2^-11. Two, as with fp32, take 172 us
// instead of 105 for 512 positions over 15k, 32 / 8 heads of 128.)
// RS: the sum of weights is of the rounded ones that the product meets, so that they add up to one and of equal values the very
// value comes out; otherwise it is of those before rounding. For fp16, whose output's step the difference reaches: that chunk is
// off by 2.24e-4 against 64 bits instead of 2.51e-4 (301 positions over 4.6k at head_dim 64 2.57e-4 and 2.69e-4), and takes 111.3 us
// instead of 105.0. A step of bf16 is eight times as wide (1.634e-3 instead of 1.638e-3): its calls keep the 6%.
template <int D, int NP, bool SC, bool RS>
__global__ void __launch_bounds__(PC8<D, NP>::THREADS, 1) attend_kernel(const Att8Args s) {
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
  // The last rows first where they see much more than the first: 8,192 positions from 0 on, 32 / 8 heads of 128, 437 us
  // instead of 449, 2,048 64 instead of 69 (but 512 over 60k 344 instead of 337).
  const int ppc = 128 / a.G, i0 = (int)(3LL * a.C > a.pos0 ? gridDim.x - 1 - blockIdx.x : blockIdx.x) * ppc;
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
  int vis_w = SC && pmax >= win_pos0 ? (int)min((int64_t)s.p.n_wsub, (pmax - win_pos0) / KW + 1) : 0;
  const int vis = vis_t + vis_w;
  const int pairs = (vis + 1) / 2;  // shares are whole pairs of blocks
  const int b0 = 2 * (int)((int64_t)pairs * share / s.p.shares);
  const int b1 = min(vis, 2 * (int)((int64_t)pairs * (share + 1) / s.p.shares));
  const int n_blk = b1 - b0;
  auto sub_of = [&](int j) { const int v = b0 + j; return !SC || v < vis_t ? v : s.p.n_tsub + (v - vis_t); };
  const uint8_t* head = a.ws + (int64_t)kvh * s.p.head_imgs * P::IMG;

  // Query rows are requested before all else. They lie apart, so that every load of a warp meets 32 lines, and what counts
  // is how few there are: 16 bytes each, kept in registers where they fit. (4,096 positions from the start, 32 / 8 heads of
  // 128, bf16: 202 us with eight bytes, twice, and results stored likewise, 169 so, 162 ahead of all else; 140 over other records.)
  constexpr int N = D / 16;  // eights of channels of half a row
  constexpr bool KEEP = N * 4 * NP <= 64;
  using Raw = Eight<NP == 2 ? KVARN_IO_F32 : KVARN_IO_F16>;  // (or bf16, which is as wide)
  Raw raw[KEEP ? N : 4]{};
  const int64_t q_at = ((int64_t)my_i * a.Hq + hq) * D + half * (D / 2);
  if (KEEP && tid < 256 && my_valid)
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i].load(a.q, q_at + 8 * i);
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
  auto query_rows = [&](auto io) {
    auto get = [&](const Raw& r, float (&x)[8]) {
      Eight<decltype(io)::value> e;
#pragma unroll
      for (int i = 0; i < NP; ++i) e.w[i] = r.w[i];
      e.get(x);
    };
    float m = 0.f;
    auto largest = [&](const Raw& r) {
      float x[8];
      get(r, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    };
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < N; ++i) largest(raw[i]);
    } else if (my_valid) {
#pragma unroll 1
      for (int i = 0; i < N; i += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) raw[k].load(a.q, q_at + 8 * (i + k));
#pragma unroll
        for (int k = 0; k < 4; ++k) largest(raw[k]);
      }
    }
    xm[half * 128 + row].x = m;
    take_over<64>(kBarPair + (warp & 3));
    const float mq = fmaxf(m, xm[(half ^ 1) * 128 + row].x), up = pow2_to(mq, 10);
    if (half == 0) xm[row].y = fabsf(a.scale) * pow2_inverse(up);
    // (maxima are taken before the positive scales; a row with an infinity becomes NaN)
    const float p2 = mq == INFINITY ? NAN : copysignf(up, a.scale);
    auto put = [&](int c0, const Raw* r) {  // 32 channels
      uint32_t hw[16], lw[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x[8];
        get(r[k], x);
#pragma unroll
        for (int i = 0; i < 8; i += 2) split_pair(x[i] * p2, x[i + 1] * p2, hw[4 * k + i / 2], lw[4 * k + i / 2]);
      }
      tmem_st16(tmem + lb + P::T_QH + half * (D / 4) + c0 / 2, hw);
      if constexpr (NP == 2 && !P::QL_SMEM) tmem_st16(tmem + lb + P::T_QL + half * (D / 4) + c0 / 2, lw);
      if constexpr (P::QL_SMEM) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(sm + sw_off(row, half * (D / 2) + c0 + 8 * k, 128)) =
              make_uint4(lw[4 * k], lw[4 * k + 1], lw[4 * k + 2], lw[4 * k + 3]);
      }
    };
    if constexpr (KEEP) {
#pragma unroll
      for (int c0 = 0; c0 < D / 2; c0 += 32) put(c0, raw + c0 / 8);
    } else {
#pragma unroll 1
      for (int c0 = 0; c0 < D / 2; c0 += 32) {
        if (my_valid)
#pragma unroll
          for (int k = 0; k < 4; ++k) raw[k].load(a.q, q_at + c0 + 8 * k);
        put(c0, raw);
      }
    }
  };
  if (tid < 256) {
    if constexpr (NP == 2) query_rows(std::integral_constant<int, KVARN_IO_F32>());
    else if (a.io == KVARN_IO_F16) query_rows(std::integral_constant<int, KVARN_IO_F16>());
    else query_rows(std::integral_constant<int, KVARN_IO_BF16>());
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
    if constexpr (SC) {
      pdl_wait();  // the scales belong to this call's images
      if (grp < n_blk) fetch_scales(grp);
    }
    auto wait = [&](uint64_t* bar, uint32_t par) { mbar_wait8(bar, par, a.err, fail); };
    int sl = grp, sl_before = 0;  // ring slot of block j and of the group's block before, and their parities
    uint32_t ph = 0, ph_before = 0;
    for (int j = grp; j < n_blk; j += NG) {
      [[maybe_unused]] float ks[NGB], lv[NGB];
      if constexpr (SC) {
#pragma unroll
        for (int g = 0; g < NGB; ++g) {
          // (not zero, so that a hidden key's -inf stays; a factor that small makes every score 0 anyway)
          ks[g] = fmaxf(ks_next[g] * qscale, 1e-37f);
          lv[g] = lv_next[g];
        }
        if (j + NG < n_blk) fetch_scales(j + NG);
      }
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
        const bool is_tile = !SC || sub < s.p.n_tsub;
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
      [[maybe_unused]] float mg[NGB];
      float ublk = -INFINITY;
      const float qs = fmaxf(qscale, 1e-37f);  // (not zero, as above)
#pragma unroll
      for (int g = 0; g < NGB; ++g) {
        float m = sv[16 * g];
#pragma unroll
        for (int u = 1; u < 15; u += 2) m = fmax3(m, sv[16 * g + u], sv[16 * g + u + 1]);
        if constexpr (SC) {
          mg[g] = fmaxf(m, sv[16 * g + 15]) * ks[g];
          ublk = fmaxf(ublk, mg[g] + lv[g]);
        } else {
          ublk = fmax3(ublk, m, sv[16 * g + 15]);
        }
      }
      if constexpr (!SC) ublk *= qs;
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
        float le = 0.f;
        if constexpr (SC) le = fmaxf(lv[g], u - fmaxf(mg[g], -1e30f) - (kHead + 50.f));
        const float kg = SC ? ks[g] : qs;
        const float2 k2 = make_float2(kg, kg), c2 = make_float2(le + kHead - u, le + kHead - u);
        float2 ls2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 x = __ffma2_rn(make_float2(sv[16 * g + 2 * e], sv[16 * g + 2 * e + 1]), k2, c2);
          const float2 w = make_float2(fast_ex2(x.x), fast_ex2(x.y));
          if constexpr (!RS) ls2 = __fadd2_rn(ls2, w);
          if constexpr (NP == 2) {
            split_pair(w.x, w.y, hw[8 * g + e], lw[8 * g + e]);
          } else {
            const __half2 h = __floats2half2_rn(w.x, w.y);
            hw[8 * g + e] = *reinterpret_cast<const uint32_t*>(&h);
            if constexpr (RS) {  // (sums of mixed types: converting back first 113.7 us instead of 111.7)
              asm("add.rn.f32.f16 %0, %1, %0;" : "+f"(ls2.x) : "h"(__half_as_ushort(__low2half(h))));
              asm("add.rn.f32.f16 %0, %1, %0;" : "+f"(ls2.y) : "h"(__half_as_ushort(__high2half(h))));
            }
          }
        }
        l_part = fmaf(ls2.x + ls2.y, SC ? fast_ex2(-le - kHead) : pow2_inverse(256.f), l_part);  // (2^-kHead)
      }
      if (SC && j >= n_t) {  // a window key's weight meets both parts of its value
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
        for (int i = 0; i < 32; ++i) v[i] *= f;
        const int c = half * (D / 2) + c0;
        // (as few stores as there can be: each of a warp's meets 32 lines)
        if (s.p.shares > 1) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) st_sector(s.acc + out_row * D + c + i, *reinterpret_cast<uint32_t(*)[8]>(v + i));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const float(&x)[8] = *reinterpret_cast<float(*)[8]>(v + i);
            if constexpr (NP == 2) Eight<KVARN_IO_F32>::store(a.out, orow * D + c + i, x);
            else if (a.io == KVARN_IO_F16) Eight<KVARN_IO_F16>::store(a.out, orow * D + c + i, x);
            else Eight<KVARN_IO_BF16>::store(a.out, orow * D + c + i, x);
          }
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
__global__ void __launch_bounds__(256) join_kernel(const Att8Args s) {
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

// Key shares of `ctas` CTAs that each see `blocks` blocks: as many as fill the SMs once. Where CTAs already fill more than
// half of them, in rounds that need not be whole, keys are shared if the rounds then cost less (WHOLE: never): a CTA takes
// as long to begin and end as 32 blocks, the join as 16 and 8 per share; kRounds rounds bound the partial results.
// (head_dim 128, bf16, 160 CTAs, us without / with shares: 63 blocks 63 / 73, 235 173 / 158, 938 623 / 464; 320 CTAs, 938
// blocks 904 / 805. At head_dim 64 158 / 136, 256 310 / 282, fp32 310 / 263 with 235 blocks.)
constexpr int kRounds = 5, kShareFrom = 128;  // (no gain with so few blocks)
template <bool WHOLE>
int key_shares(int64_t ctas, int64_t blocks) {
  const int64_t sms = sm_count();
  int64_t shares = ctas > 0 ? sms / ctas : 1;
  const int64_t most = blocks / 4;  // two pairs of blocks per share at least
  if (shares > most) shares = most;
  if (shares > 64) shares = 64;
  if (shares < 1) shares = 1;
  if (WHOLE || 2 * ctas <= sms || blocks <= kShareFrom) return (int)shares;
  double least = 0;
  for (int64_t n = 1; n * ctas <= kRounds * sms || n == 1; ++n) {
    const double cost = (double)((n * ctas + sms - 1) / sms) * ((double)blocks / n + 32) + (n > 1 ? 16 + 8 * n : 0);
    if (n == 1 || cost < least) {
      least = cost;
      shares = n;
    }
  }
  return (int)shares;
}

// Workspace of a call over n_tblk tiles and win_vis window rows, with or without scales.
Plan8 plan8(int C, int n_tblk, int win_vis, int Hq, int Hkv, int D, bool fp32, bool scaled) {
  Plan8 p;
  const int KB = PC8<64, 1>::KB, G = Hq / Hkv, ppc = 128 / G;
  p.n_tsub = n_tblk * (kTile / KB);
  p.n_wsub = (win_vis + 2 * PC8<64, 1>::KW - 1) / (2 * PC8<64, 1>::KW) * 2;
  p.head_imgs = 2LL * (p.n_tsub + p.n_wsub);
  p.row_blocks = (int)(((int64_t)C + ppc - 1) / ppc);
  const int64_t ctas = (int64_t)p.row_blocks * Hkv;
  p.shares = scaled ? key_shares<true>(ctas, p.n_tsub + p.n_wsub) : key_shares<false>(ctas, p.n_tsub);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p.off_scale = up((size_t)Hkv * p.head_imgs * KB * D * 2);
  p.off_ml = p.off_scale + (scaled ? up((size_t)Hkv * (p.n_tsub + p.n_wsub) * 64) : 0);
  const size_t rows = p.shares > 1 ? (size_t)p.shares * C * Hq : 0;
  p.off_acc = p.off_ml + up(rows * sizeof(float2));
  p.off_sum = p.off_acc + up(rows * D * sizeof(float));
  const bool emptied = fp32 && p.n_tsub + p.n_wsub > kEmpty;
  p.bytes = p.off_sum + (emptied ? up((size_t)ctas * p.shares * 128 * D * sizeof(float)) : 0);
  return p;
}

// The attention kernel behind the grid that makes the images, and the join.
template <int D, int NP, bool SC, bool RS>
cudaError_t launch_attend(const Att8Args& s, cudaStream_t st) {
  using P = PC8<D, NP>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(attend_kernel<D, NP, SC, RS>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  LaunchCfg L(dim3(s.p.row_blocks, s.a.Hkv, s.p.shares), dim3(P::THREADS), P::SMEM, st, KVARN_LAUNCH_PDL);
  e = cudaLaunchKernelEx(&L.cfg, attend_kernel<D, NP, SC, RS>, s);
  if (e != cudaSuccess || s.p.shares == 1) return e;
  const int64_t rows = (int64_t)s.a.C * s.a.Hq;
  LaunchCfg J(dim3((unsigned)((rows + 1024 / D - 1) / (1024 / D))), dim3(256), 0, st, KVARN_LAUNCH_PDL);
  return cudaLaunchKernelEx(&J.cfg, join_kernel<D>, s);
}

}  // namespace
}  // namespace kvarn
