// decode4.cu -- single-token attention over 4-bit records.
//
//   split kernel   The tiles of all (sequence, KV head) segments, one after another, are cut into one equal share per
//                  CTA, by the lengths that the device holds: ragged batches keep every SM busy to the end. A CTA of four
//                  warps works through its share; its warp w takes the run w (32 tokens) of each tile, streams it by
//                  bulk copies of its own and keeps a softmax of its own. The four meet at the end of a piece (a share's
//                  part of a segment), and the piece's maximum m, sum l and accumulator (in units of 2^m) go to
//                  the workspace, in the slot CTA + segment.
//   merge kernel   joins the pieces of a head, found by the same arithmetic, and, on request, adds up tiles' weights.
//
// Short tables need neither: a CTA takes a segment by itself, several tiles side by side, and writes its rows and weights.
//
// The warps need no exchange while they run because a run's scores and values both stay in one warp: the codes
// become fp16 numbers in registers, exactly (unit_values), as the A operand of mma.sync m16n8k16, for the scores
// (16 tokens x 16 channels) and, read transposed, for the values (16 channels x 16 tokens). Queries and
// probabilities are the other operand, as pairs hi + lo of fp16 (22 bits). Its eight columns are
//   up to four heads to a group   a head's hi and lo part in neighbouring columns: one product for both, whose
//                                 results a lane adds, and none spent on padding
//   more (WIDE)                   eight heads, the parts in products of their own. A 16-bit query needs no lo part.
// Probabilities go from the first product's result to the second one's operand by movmatrix.
//   s_t = (q . k_t) scale,   O = O 2^(M_old - M) + sum_t 2^(s_t - M) v_t, the sum of a run in accumulators of its own
// (the tensor core drops what falls below a sum's last bit), joined to O with rounding.
//
// What bounds it: HBM in batches (32 ragged sequences of up to 32k tokens, head_dim 256, 755 MB in 120 us: 6.3 TB/s, 92%
// of the measured copy rate), instructions otherwise: 2.4 per code at head_dim 128, of which 1.4 unpack it (four
// sequences of 64k tokens, 302 MB in 58.3 us, 5.2 TB/s, at 2.6 instructions per cycle of 4; head_dim 64 3.9 TB/s in 38.7
// us; groups of eight heads 3.7 TB/s). Short calls are a chain of latencies: length, table, copy, exchange, merge (4 tiles
// 5.5 us; 16k tokens 10.2 against 2.8 of bytes). On the way from 172.7 us for the batch: run-time mask base (142),
// shares by actual lengths instead of items of a fixed span (127), the merge's arithmetic ahead of its wait and typed
// query loads (120). Not kept: two runs to a step (fewer exchanges, but fewer warps: 81 us against 74 at the time),
// three or four runs in flight per warp, 20 warps per SM at head_dim 128 (96 registers: 60.9 against 58.5).
//
// The same kernels serve chunks of a few positions (CHUNK): eight (position, head) rows to a segment, each of which
// sees the cache up to its own position.
#include <type_traits>

#include "cache4.cuh"
#include "join.cuh"

namespace kvarn {
namespace {

constexpr float kNone = -3.0e38f;  // reference exponent before the first run
constexpr float kHead = 14.f;      // probabilities reach 2^14: lo parts stay normal fp16 numbers

// TW: tiles that a CTA's warps take side by side; more than one in the kernel that does a segment by itself.
template <int D_, bool WIDE, int TW = 1>
struct C4 {
  static constexpr int D = D_;
  static constexpr int NW = kRuns * TW;        // warps, one per run of a tile
  static constexpr int HL = WIDE ? 2 : 1;      // rows (heads) whose scores a lane holds
  static constexpr int ROWS = 4 * HL;
  // Runs of a warp under way or in use: two keep some 70 KB per SM in flight, and more were no faster (four sequences of
  // 64k tokens, head_dim 128: 58.5 us with two and four CTAs, 59.9 with three and four, 58.8 with three and three).
  static constexpr int STG = 2;
  // CTAs resident per SM: what registers allow without spilling, or a little fewer (two of six-head groups at head_dim
  // 64: 17.6 us with four, 18.2 with three; 120 us of batched decode at head_dim 256 with three, 126 with two).
  static constexpr int CTAS = TW > 1 ? 1 : D == 64 ? 4 : D == 128 ? (WIDE ? 3 : 4) : WIDE ? 2 : 3;
  static constexpr int RB = Run4<D>::kBytes;
  static constexpr int OS = D + 8;             // floats of a row where the warps meet
  static constexpr int OFF_ML = NW * STG * RB; // float2 [NW][8]: (m, l)
  static constexpr int OFF_BAR = OFF_ML + NW * 64;
  static constexpr int OFF_FLG = OFF_BAR + 8 * NW * STG;
  static constexpr int SMEM = (OFF_FLG + 8 + 127) / 128 * 128;
  static_assert(ROWS * OS * 4 <= STG * RB, "a warp's accumulators fit in its ring");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same product on its own.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// 8 x 8 matrix of 16-bit elements, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Reads of shared memory at a 32-bit address: bases are formed once per run, the rest is in the instruction.
__device__ __forceinline__ void load_transposed(uint32_t p, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(p)
               : "memory");
}
__device__ __forceinline__ void load16(uint32_t p, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(p) : "memory");
}
__device__ __forceinline__ void load8(uint32_t p, uint32_t (&v)[2]) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(p) : "memory");
}
__device__ __forceinline__ __half load_half(uint32_t p) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
  return __ushort_as_half(v);
}

struct Split4Args {
  Decode4Args a;
  float2* ml;       // [slots][rows of a CTA]
  float* acc;       // [slots][rows of a CTA][D]
  float2* tile_ml;  // [B][Hkv][max_tiles][4][8], or NULL
  int ctas, few;    // see Shares4
  uint32_t base;    // kUnitBase
  int pos0, n_tiles;  // CHUNK: B positions of one sequence instead of B sequences
};

// Score row r (0..7) of a segment: with CHUNK the (position, head) pairs of a KV head, eight to a segment, are rows of one
// sequence that see the cache up to their own position; otherwise the G heads of sequence b.
struct Row4 {
  bool valid;
  int64_t index;  // among the rows of queries and outputs
  int seen;       // cached tokens that the row sees
};
template <bool CHUNK>
__device__ __forceinline__ Row4 row4(const Split4Args& s, int b, int kvh, int r) {
  const Decode4Args& a = s.a;
  if constexpr (CHUNK) {
    const int64_t n = 8LL * b + r, i = n / a.G;
    const bool valid = i < a.B;
    return Row4{valid, valid ? i * a.Hq + (int64_t)kvh * a.G + n % a.G : 0, valid ? s.pos0 + (int)i + 1 : 0};
  } else {
    return Row4{r < a.G, (int64_t)b * a.Hq + (int64_t)kvh * a.G + min(r, a.G - 1), INT32_MAX};
  }
}

// Cached tokens of sequence b, and the tiles that hold them; of a CHUNK's rows 8 b .. 8 b + 7 what any of them sees,
// and of tiles the same number for all, so that places need no sums.
template <bool CHUNK>
__device__ __forceinline__ int tokens4(const Split4Args& s, int b) {
  if constexpr (CHUNK) return s.pos0 + min(s.a.B, (8 * b + 7) / s.a.G + 1);
  else return min(max(s.a.lens[b], 0), kTile * s.a.max_tiles);
}
template <bool CHUNK>
__device__ __forceinline__ int tiles4(const Split4Args& s, int b) {
  if constexpr (CHUNK) return s.n_tiles;
  else return (tokens4<CHUNK>(s, b) + kTile - 1) / kTile;
}
// Shares of `total` tiles, at most one per resident CTA; the first `more` of them hold base + 1 tiles, the others base,
// so that none is empty and a segment's pieces lie in slots side by side. A share costs a CTA as much as two tiles
// besides (query, exchange, partial result), so there are three tiles to one, where that leaves `few` (two CTAs per
// SM): one sequence of 16k tokens took 10.7 us so (10.2 now), with a share per CTA 11.6, with four tiles to a share 11.9; 4k
// 6.5 with one tile, 7.0 with two. (All counts are below 2^31: 64-bit divisions would take a microsecond of a
// short call.)
struct Shares4 {
  int total, n, base, more;
  __device__ __forceinline__ Shares4(int total_, int ctas, int few) : total(total_) {
    n = min(ctas, max(min(total, few), total / 3));
    base = total / max(n, 1);
    more = total - base * n;
  }
  __device__ __forceinline__ int begin(int c) const { return c < n ? c * base + min(c, more) : total; }
  __device__ __forceinline__ int of(int u) const {  // the share that tile u belongs to
    const int wide = more * (base + 1);
    return u < wide ? u / (base + 1) : more + (u - wide) / base;
  }
};

// What a CTA needs to know of all sequences: the tiles before sequence `want` (per KV head) and in all of them; or,
// with want < 0, the sequence that tile at(total) lies in. One pass over the lengths, a run of them per thread.
// Every thread of the CTA gets the answer; scratch: 2 + warps words of shared memory.
struct Before4 {
  int total, before;  // in tiles of one KV head
  int b;
};
template <int THREADS, class At>
__device__ __forceinline__ Before4 before4(const Split4Args& s, int want, At at, int* scratch) {
  const int B = s.a.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (B == 1) return Before4{tiles4<false>(s, 0), 0, 0};
  const int per = (B + THREADS - 1) / THREADS, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles4<false>(s, b);
  int upto = mine;  // inclusive sum over the warp's threads
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, m);
    if (lane >= m) upto += x;
  }
  if (lane == 31) scratch[2 + warp] = upto;
  __syncthreads();
  int total = 0, first = upto - mine;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) first += scratch[2 + w];
    total += scratch[2 + w];
  }
  const int u = want < 0 ? at(total) : 0;
  for (int b = b0; b < b1; ++b) {
    const int n = per == 1 ? mine : tiles4<false>(s, b);
    if (want < 0 ? u >= first && u < first + n : b == want) {
      scratch[0] = first;
      scratch[1] = b;
    }
    first += n;
  }
  __syncthreads();
  return Before4{total, scratch[0], scratch[1]};
}

// NQ: parts of a query in WIDE products, 1 for 16-bit ones. TW > 1: a CTA does segment (KV head blockIdx.x, blockIdx.y)
// by itself and writes its output.
template <int D, bool WIDE, int NQ, bool CHUNK, int TW>
__global__ void __launch_bounds__(32 * C4<D, WIDE, TW>::NW, C4<D, WIDE, TW>::CTAS) split4_kernel(const Split4Args s) {
  using C = C4<D, WIDE, TW>;
  constexpr bool ALONE = TW > 1;
  using R = Run4<D>;
  constexpr int STG = C::STG, RB = C::RB, HL = C::HL;
  constexpr int BLK = D / R::kWide;        // blocks of K units
  constexpr int WPB = R::kWide / 32;       // words (8 channels) of a token that a lane holds, per block
  extern __shared__ __align__(128) unsigned char smem[];
  const Decode4Args& a = s.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int part = warp % kRuns;  // the run of a tile that is this warp's
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * STG;
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLG);
  unsigned char* ring = smem + warp * STG * RB;
  if (tid == 0) *flag = 0;
  if (lane == 0) {
    for (int i = 0; i < STG; ++i) mbar_init_n(bar + i, 1);
    mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();
  // this CTA's share, and the segment and tile that it begins with
  int now, end, b, kvh = 0, tile0 = 0;
  if constexpr (ALONE) {
    b = blockIdx.y;
    kvh = blockIdx.x;
    now = 0;
    end = tiles4<CHUNK>(s, b);
  } else {
    auto begin_in = [&](int t) {  // (with no share: nowhere)
      const Shares4 x(t * a.Hkv, s.ctas, s.few);
      return (int)blockIdx.x < x.n ? x.begin(blockIdx.x) / a.Hkv : -1;
    };
    Before4 at;
    if constexpr (CHUNK) {
      at.total = (int)(((int64_t)a.B * a.G + 7) / 8) * s.n_tiles;
      at.b = max(begin_in(at.total), 0) / s.n_tiles;
      at.before = at.b * s.n_tiles;
    } else {
      at = before4<128>(s, -1, begin_in, reinterpret_cast<int*>(smem));  // (the rings are still unused)
    }
    const Shares4 x(at.total * a.Hkv, s.ctas, s.few);
    now = x.begin(blockIdx.x);
    end = x.begin(blockIdx.x + 1);
    b = at.b;
    if (now < end) {
      const int n = tiles4<CHUNK>(s, b), in = now - at.before * a.Hkv;
      kvh = in / n;
      tile0 = in - kvh * n;
    }
  }
  if (!ALONE && now >= end) return;  // (a segment of no tokens passes through)
  if (ALONE) {
    __syncthreads();  // (the flag)
  } else if (!CHUNK && a.B > 1) {  // the scratch words go back to the copies
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  bool ok = true;
  int sl = 0;  // slot of the next run, and the parity of its use
  uint32_t use = 0;
  unsigned bad = 0;  // bit i: the run in slot i has no record
#pragma unroll 1
  for (;;) {  // piece by piece
    const int first = tile0, len = tokens4<CHUNK>(s, b);
    const int nt = min(tiles4<CHUNK>(s, b) - first, end - now);
    const int stop = first + nt;
    const int64_t* table = a.tile_table + ((CHUNK ? 0 : (int64_t)b * a.Hkv) + kvh) * a.max_tiles + first;
    // This warp's tiles are first + tw, and every TW-th after it. Runs of 32 of them, one address per lane, NULL for one that
    // does not lie in the pool.
    const int tw = warp / kRuns;
    auto address = [&](int j) -> const uint8_t* {
      if (first + tw + j * TW >= stop) return nullptr;
      const int64_t off = table[tw + j * TW];
      return (off & 15) || off < 0 || off > a.tiles_bytes - R::kRecord ? nullptr : a.tiles + off + part * RB;
    };
    const uint8_t* source = address(lane);
    constexpr int kStep = kTile * TW;                            // tokens from one of this warp's runs to the next
    const int run0 = kTile * (first + tw) + kRun * part;         // first token of this warp
    // runs of this warp that hold tokens
    const int nr = max((int)((min((int64_t)len, (int64_t)kTile * stop) - run0 + kStep - 1) / kStep), 0);
    __syncwarp();
    auto request = [&](int j, int sl) {
      if (j >= nr) return;
      const uint64_t src = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(source), j & 31);
      bad &= ~(1u << sl);
      if (src == 0) bad |= 1u << sl;
      if (lane == 0) {
        if (src == 0) {
          report(a.err, KVARN_DEVERR_RECORD);
          mbar_arrive1(bar + sl);
        } else {
          mbar_arrive_tx(bar + sl, RB);
          bulk_in(ring + sl * RB, reinterpret_cast<const uint8_t*>(src), RB, bar + sl);
        }
      }
    };
    auto next_slot = [&](int x) { return x + 1 == STG ? 0 : x + 1; };
    for (int j = 0, x = sl; j < STG; ++j, x = next_slot(x)) request(j, x);

    // B fragments of the query. Column g: part g % 2 of row g / 2, or (WIDE) row g, its parts in qb[0] and qb[1]. A
    // product's channels are those that a word of K units gives to two registers.
    uint32_t qb[NQ][BLK * WPB][4];
    float c1[HL];             // of the rows whose scores this lane holds: HL q + 0 ..
    [[maybe_unused]] int seen[HL];
    {
      const Row4 me = row4<CHUNK>(s, b, kvh, WIDE ? g : g >> 1);
      float x[BLK * WPB][8];
      float mx = 0.f;
      auto load = [&](auto io) {  // (loads of a type that is known: under way together)
        Eight<decltype(io)::value> e[BLK * WPB];
#pragma unroll
        for (int w = 0; w < BLK * WPB; ++w)
          e[w].load(a.q, me.index * D + w / WPB * R::kWide + q * (R::kWide / 4) + 8 * (w % WPB));
#pragma unroll
        for (int w = 0; w < BLK * WPB; ++w) {
          e[w].get(x[w]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!me.valid) x[w][i] = 0.f;
            mx = fmaxf(mx, fabsf(x[w][i]));
          }
        }
      };
      if (a.io == KVARN_IO_F32) load(std::integral_constant<int, KVARN_IO_F32>());
      else if (a.io == KVARN_IO_F16) load(std::integral_constant<int, KVARN_IO_F16>());
      else load(std::integral_constant<int, KVARN_IO_BF16>());
      mx = fmaxf(mx, shfl_xor(mx, 1));
      mx = fmaxf(mx, shfl_xor(mx, 2));
      // (a row with an infinity becomes NaN: without a lo part its scores could be infinite)
      const float p2 = mx == INFINITY ? NAN : pow2_to(mx, 10);
#pragma unroll
      for (int w = 0; w < BLK * WPB; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t hi, lo;
          split_pair(x[w][j] * p2, x[w][j + 4] * p2, hi, lo);
          qb[0][w][j] = !WIDE && (g & 1) ? lo : hi;
          if constexpr (NQ == 2) qb[1][w][j] = lo;
        }
      const float c = a.scale * pow2_inverse(pow2_to(mx, 10));
#pragma unroll
      for (int h = 0; h < HL; ++h) {
        c1[h] = __shfl_sync(0xffffffffu, c, 8 * q + 4 * h);  // (column 2 q, or 2 q + h)
        if constexpr (CHUNK) seen[h] = row4<CHUNK>(s, b, kvh, HL * q + h).seen;
      }
    }

    float M[HL], l[HL];
    float o[D / 16][2][HL];
#pragma unroll
    for (int h = 0; h < HL; ++h) {
      M[h] = kNone;
      l[h] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][0][h] = o[i][1][h] = 0.f;
    }
    const uint32_t ring_at = smem_addr(ring);
    // this lane's places in a run: K units and scales of token g, V units, V scales
    const uint32_t at_k = ring_at + g * (R::kWide / 2) + q * (R::kWide / 8);
    const uint32_t at_ks = ring_at + R::kKScale + 2 * (g * R::kGroups + (WPB == 4 ? q : q >> 1));
    const uint32_t at_v = ring_at + R::kVCodes + lane * 16, at_vs = ring_at + R::kVScale + q * 16;
    // run j, which lies in slot sl; EDGE: some of its tokens are not seen, or it has no record
    auto work_on = [&](int j, auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
      const uint32_t run = sl * RB;
      const int n_tok = len - run0 - kStep * j;  // tokens from the run's first on
      const bool none = bad >> sl & 1;
      // scores of tokens 8 x + g of the run for row HL q + h
      float sc[HL][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float e[2][4];  // sums of their own for every other product
#pragma unroll
        for (int k = 0; k < BLK; ++k) {
          uint32_t kw[2][WPB];
          __half2 ks[2], kt[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int t = 16 * mt + 8 * r;
            const uint32_t p = at_k + run + (k * (kRun * R::kWide / 2) + t * (R::kWide / 2));
            if constexpr (WPB == 4) load16(p, kw[r]);
            else load8(p, kw[r]);
            ks[r] = __half2half2(load_half(at_ks + run + 2 * (t * R::kGroups + 4 * k)));
            kt[r] = minus24(ks[r]);
          }
#pragma unroll
          for (int w = 0; w < WPB; ++w) {
            uint32_t x[2][4];
            unit_values(kw[0][w], ks[0], kt[0], s.base, x[0]);
            unit_values(kw[1][w], ks[1], kt[1], s.base, x[1]);
#pragma unroll
            for (int p = NQ - 1; p >= 0; --p) {  // (the lo parts first, while the sums are small)
              const uint32_t (&f)[4] = qb[p][k * WPB + w];
              if (k == 0 && w == 0 && p == NQ - 1) {
                mma_f16_new(e[0], x[0][0], x[1][0], x[0][1], x[1][1], f[0], f[1]);
                mma_f16_new(e[1], x[0][2], x[1][2], x[0][3], x[1][3], f[2], f[3]);
              } else {
                mma_f16(e[0], x[0][0], x[1][0], x[0][1], x[1][1], f[0], f[1]);
                mma_f16(e[1], x[0][2], x[1][2], x[0][3], x[1][3], f[2], f[3]);
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < HL; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            sc[h][2 * mt + r] = (WIDE ? e[0][2 * r + h] + e[1][2 * r + h]
                                      : (e[0][2 * r] + e[1][2 * r]) + (e[0][2 * r + 1] + e[1][2 * r + 1])) * c1[h];
      }
      if constexpr (EDGE) {
#pragma unroll
        for (int h = 0; h < HL; ++h)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (none) sc[h][x] = NAN;
            if (8 * x + g >= (CHUNK ? seen[h] - run0 - kStep * j : n_tok)) sc[h][x] = -INFINITY;
          }
      }
      float alpha[HL], p[HL][4];
#pragma unroll
      for (int h = 0; h < HL; ++h) {
        float m = fmaxf(fmaxf(sc[h][0], sc[h][1]), fmaxf(sc[h][2], sc[h][3]));
        m = fmaxf(m, shfl_xor(m, 4));
        m = fmaxf(m, shfl_xor(m, 8));
        m = fmaxf(m, shfl_xor(m, 16));
        m = fmaxf(m - kHead, M[h]);
        alpha[h] = fast_ex2(M[h] - m);
        M[h] = m;
#pragma unroll
        for (int x = 0; x < 4; ++x) p[h][x] = fast_ex2(sc[h][x] - m);
        float sum = (p[h][0] + p[h][1]) + (p[h][2] + p[h][3]);
        l[h] = fmaf(l[h], alpha[h], sum);
        if (s.tile_ml) {  // the run's part of its tile's weight
          sum += shfl_xor(sum, 4);
          sum += shfl_xor(sum, 8);
          sum += shfl_xor(sum, 16);
          if (g == 0)
            s.tile_ml[((((int64_t)b * a.Hkv + kvh) * a.max_tiles + first + tw + j * TW) * kRuns + part) * 8 + HL * q + h] =
                make_float2(m, sum);
        }
      }
      // B fragments of the probabilities, by tokens 8 x .. 8 x + 7
      uint32_t pb[HL][4];
      if constexpr (WIDE) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t hi, lo;
          split_pair(p[0][x], p[1][x], hi, lo);
          pb[0][x] = transpose8(hi);
          pb[1][x] = transpose8(lo);
        }
      } else {
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          uint32_t hi, lo;
          split_pair(p[0][x], p[0][x + 1], hi, lo);
          pb[0][x] = transpose8(__byte_perm(hi, lo, 0x5410));
          pb[0][x + 1] = transpose8(__byte_perm(hi, lo, 0x7632));
        }
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[4], vs[4];
        load_transposed(at_v + run + c * 512, v);
        load16(at_vs + run + c * 64, vs);
        if constexpr (EDGE) {  // what lies behind the last token counts as zeros, whatever it is
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int t = 8 * x + 2 * q;
            vs[x] &= none || t >= n_tok ? 0u : t + 1 < n_tok ? 0xFFFFFFFFu : 0x0000FFFFu;
          }
        }
        uint32_t x[4][4];  // [8 tokens][channel]
#pragma unroll
        for (int t = 0; t < 4; ++t) unit_values(v[t], as_half2(vs[t]), minus24(as_half2(vs[t])), s.base, x[t]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // channels 32 c + 4 g + 2 i and the next, in rows g and g + 8
          float d[4];
#pragma unroll
          for (int h = HL - 1; h >= 0; --h) {  // (WIDE: the lo parts, then the hi parts)
            if (h == HL - 1) mma_f16_new(d, x[0][2 * i], x[0][2 * i + 1], x[1][2 * i], x[1][2 * i + 1], pb[h][0], pb[h][1]);
            else mma_f16(d, x[0][2 * i], x[0][2 * i + 1], x[1][2 * i], x[1][2 * i + 1], pb[h][0], pb[h][1]);
            mma_f16(d, x[2][2 * i], x[2][2 * i + 1], x[3][2 * i], x[3][2 * i + 1], pb[h][2], pb[h][3]);
          }
          float (&y)[2][HL] = o[2 * c + i];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < HL; ++h)
              y[r][h] = fmaf(y[r][h], alpha[h], WIDE ? d[2 * r + h] : d[2 * r] + d[2 * r + 1]);
        }
      }
    };
    // tokens that every row sees
    const int whole = CHUNK ? s.pos0 + 8 * b / a.G + 1 : len;
#pragma unroll 1
    for (int j = 0; j < nr; ++j) {
      ok &= mbar_wait8(bar + sl, use, a.err);
      if ((bad >> sl & 1) || whole - run0 - kStep * j < kRun) work_on(j, std::true_type());
      else work_on(j, std::false_type());
      __syncwarp();  // the slot is used up
      const int ahead = j + STG;
      if ((ahead & 31) == 0 && ahead < nr) source = address(ahead + lane);
      request(ahead, sl);
      sl = next_slot(sl);
      if (sl == 0) use ^= 1;
    }
    if (!ok) {  // a copy whose wait ran out still writes to this CTA's memory: each is given as long again
      *flag = 1;
      for (int i = 0; i < STG; ++i) mbar_wait8(bar + i, i < sl ? use : use ^ 1, nullptr);
    }
    if (s.tile_ml && g == 0)  // runs of the last tile that hold nothing
      for (int j = nr; tw + j * TW < nt; ++j)
#pragma unroll
        for (int h = 0; h < HL; ++h)
          s.tile_ml[((((int64_t)b * a.Hkv + kvh) * a.max_tiles + first + tw + j * TW) * kRuns + part) * 8 + HL * q + h] =
              make_float2(kNone, 0.f);
    // the warps meet: each leaves its rows in its own ring
    float* mine = reinterpret_cast<float*>(ring);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < HL; ++h) {
      l[h] += shfl_xor(l[h], 4);
      l[h] += shfl_xor(l[h], 8);
      l[h] += shfl_xor(l[h], 16);
      if (g == 0) ml[warp * 8 + HL * q + h] = make_float2(nr > 0 ? M[h] : -INFINITY, l[h]);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<float2*>(mine + (HL * q + h) * C::OS + 32 * (i / 2) + 4 * g + 2 * (i % 2)) =
            make_float2(o[i][0][h], o[i][1][h]);
    }
    __syncthreads();
    const bool lost = *flag != 0;
    if (ALONE && lost) {
      if (tid < 8) ml[tid].y = NAN;
      __syncthreads();
    }
    const int64_t slot = blockIdx.x + (int64_t)b * a.Hkv + kvh;
    for (int i = tid; i < C::ROWS * (D / 4); i += 32 * C::NW) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      const Row4 me = row4<CHUNK>(s, b, kvh, r);
      if (!me.valid) continue;
      float2 v[C::NW];
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        v[w] = ml[w * 8 + r];
        m = fmaxf(m, v[w].x);
      }
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        const float f = v[w].x == -INFINITY ? 0.f : fast_ex2(v[w].x - m);
        const float4 x = *reinterpret_cast<const float4*>(smem + w * STG * RB + (r * C::OS + c) * 4);
        sum = fmaf(f, v[w].y, sum);
        y.x = fmaf(f, x.x, y.x); y.y = fmaf(f, x.y, y.y); y.z = fmaf(f, x.z, y.z); y.w = fmaf(f, x.w, y.w);
      }
      if constexpr (ALONE) {
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        io_st4(a.out, a.io, me.index * D + c, make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
        continue;
      }
      *reinterpret_cast<float4*>(s.acc + (slot * C::ROWS + r) * D + c) = y;
      if (c == 0) s.ml[slot * C::ROWS + r] = lost ? make_float2(0.f, NAN) : make_float2(m, sum);
    }
    if constexpr (ALONE) {
      if (a.mass_out) {  // (the tiles' parts lie behind the barrier too)
        const int64_t at = ((int64_t)b * a.Hkv + kvh) * a.max_tiles;
        join_masses<kRuns, 8>(ml, 1, C::NW, s.tile_ml + at * kRuns * 8, a.G, 0, nt, a.max_tiles,
                              a.mass_in ? a.mass_in + at : nullptr, a.mass_out + at);
      }
      break;
    }
    now += nt;
    if (now >= end) break;
    // the next segment that holds tiles; the rings go back to the copies
    tile0 = 0;
    if (++kvh == a.Hkv) {
      kvh = 0;
      do ++b;
      while (tiles4<CHUNK>(s, b) == 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
}

// Joins the pieces of a segment's rows (EACH: those of query head blockIdx.x of row block blockIdx.y, a sequence or a position
// of a CHUNK; else all of KV head blockIdx.x), or adds up the weights of 256 tiles of a KV head.
template <int D, int ROWS, bool CHUNK, bool EACH>
__global__ void __launch_bounds__(256) merge4_kernel(const Split4Args s, int mass_blocks) {
  const Decode4Args& a = s.a;
  __shared__ int scratch[10];
  const int joins = EACH ? a.Hq : a.Hkv;
  const bool mass = (int)blockIdx.x >= joins;
  const int kvh = mass ? ((int)blockIdx.x - joins) / mass_blocks : EACH ? (int)blockIdx.x / a.G : (int)blockIdx.x;
  const int64_t n = EACH && CHUNK ? (int64_t)blockIdx.y * a.G + blockIdx.x % a.G : 0;  // row among a CHUNK's of this KV head
  const int b = EACH && CHUNK ? (int)(n / 8) : blockIdx.y;
  pdl_trigger();
  // (the lengths are not the split kernel's: they have been there since before its first CTA let this kernel start)
  Before4 at;
  if constexpr (CHUNK) at = Before4{(int)(((int64_t)a.B * a.G + 7) / 8) * s.n_tiles, b * s.n_tiles, b};
  else at = before4<256>(s, b, [](int) { return 0; }, scratch);
  const int tiles = tiles4<CHUNK>(s, b), u = at.before * a.Hkv + kvh * tiles;
  const Shares4 x(at.total * a.Hkv, s.ctas, s.few);
  const int c = tiles ? x.of(u) : 0, pieces = tiles ? x.of(u + tiles - 1) - c + 1 : 0;
  const int64_t slot = (c + (int64_t)b * a.Hkv + kvh) * ROWS;
  pdl_wait();
  if (mass) {
    const int64_t first = ((int64_t)b * a.Hkv + kvh) * a.max_tiles;
    join_masses<kRuns, ROWS>(s.ml + slot, 1, pieces, s.tile_ml + first * kRuns * 8, a.G,
                             ((int)blockIdx.x - joins) % mass_blocks, tiles, a.max_tiles,
                             a.mass_in ? a.mass_in + first : nullptr, a.mass_out + first);
  } else if constexpr (EACH) {
    const int r = CHUNK ? (int)(n % 8) : (int)blockIdx.x % a.G;
    join_items<D, ROWS>(s.ml + slot + r, s.acc + (slot + r) * D, pieces, a.out, a.io, (int64_t)blockIdx.y * a.Hq + blockIdx.x);
  } else if (pieces <= 32) {  // (more where most sequences are empty)
    const int r = threadIdx.x / 32;
    const Row4 me = row4<CHUNK>(s, b, kvh, r);
    if (r < ROWS && me.valid) join_few<D, ROWS>(s.ml + slot + r, s.acc + (slot + r) * D, pieces, a.out, a.io, me.index);
  } else {
    for (int r = 0; r < ROWS; ++r) {
      const Row4 me = row4<CHUNK>(s, b, kvh, r);
      if (me.valid) join_items<D, ROWS>(s.ml + slot + r, s.acc + (slot + r) * D, pieces, a.out, a.io, me.index);
      __syncthreads();
    }
  }
}

template <class Kernel>
cudaError_t allow_shared(Kernel* kernel, int bytes, bool (&configured)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) configured[dev] = true;
  }
  return e;
}

// Tiles that a CTA takes side by side when it does a segment by itself: 16 warps, or 8 that need more registers. One launch and
// no partial results, so short tables are read by it: of kAloneChannels tiles x channels at most, or of up to 4 TW tiles where
// there are two segments to five SMs. An SM holds one such CTA, and nothing covers the ends and beginnings of CTAs one after another: in
// a second round tables are of 2 TW tiles at most, and more segments than two rounds of them are shared out like long tables. Both
// ways, in us (joined pieces / by itself), bf16 queries, full tables:
//   D 64, G 4     8 segments: 2 tiles 5.4 / 3.9, 6 5.5 / 5.4, 8 5.5 / 6.0;   64: 4 7.2 / 5.0, 16 9.8 / 8.4
//                 304: 4 11.1 / 8.6, 8 11.3 / 11.0, 16 15.8 / 15.9;   512: 4 13.3 / 15.2;   2,048: 1 26.0 / 36.5, 6 47.8 / 68.0
//   D 128, G 4    8: 2 6.0 / 5.0, 3 5.9 / 5.4, 4 5.9 / 6.0;   64: 4 8.0 / 6.2, 16 12.3 / 11.6
//                 304: 4 13.9 / 11.3, 8 14.8 / 15.4, 16 22.2 / 23.3;   512: 4 16.9 / 20.5;   2,048: 1 30.0 / 48.6, 6 65.9 / 93.2
//   D 128, G 8    8: 1 6.1 / 4.5, 3 6.2 / 6.0, 4 6.2 / 6.4;   64: 4 8.0 / 6.6, 8 10.1 / 9.3;   304: 4 14.8 / 12.1;   2,048: 3 54.6 / 74.6
//   D 256, G 4    8: 1 7.5 / 5.7, 2 7.5 / 6.2, 3 7.3 / 7.7;   64: 4 10.1 / 8.1, 8 11.6 / 11.7;   304: 4 20.0 / 15.6;   2,048: 4 92.9 / 102.6
// Over 960 sizes (8 to 2,048 segments, 1 to 16 tiles, full and ragged) the choice costs 1.2% on the mean, 35% at worst.
constexpr int kAloneChannels = 384;
template <int D, bool WIDE>
constexpr int kSideBySide = D == 64 || (D == 128 && !WIDE) ? 4 : 2;  // (16 warps, or 8 that need the registers)

template <int D, bool WIDE, int NQ, bool CHUNK>
cudaError_t launch_d4(const Decode4Plan& p, Split4Args& s, void* ws, cudaStream_t st) {
  const Decode4Args& a = s.a;
  unsigned char* w = static_cast<unsigned char*>(ws);
  s.base = kUnitBase;
  s.tile_ml = a.mass_out ? reinterpret_cast<float2*>(w + p.off_tile) : nullptr;
  constexpr int TW = kSideBySide<D, WIDE>;
  const int tiles = CHUNK ? s.n_tiles : a.max_tiles;
  const int64_t blocks = CHUNK ? ((int64_t)a.B * a.G + 7) / 8 : a.B;  // of sequences, or of eight rows
  const int64_t segments = blocks * a.Hkv, sms = sm_count();
  // (tables of no tiles, which would make no shares, among them)
  if (segments <= sms ? (int64_t)tiles * D <= kAloneChannels || (tiles <= 4 * TW && 5 * segments >= 2 * sms)
                      : tiles == 0 || (segments <= 2 * sms && tiles <= 2 * TW)) {
    using C = C4<D, WIDE, TW>;
    static bool configured[64] = {};
    cudaError_t e = allow_shared(split4_kernel<D, WIDE, NQ, CHUNK, TW>, C::SMEM, configured);
    if (e != cudaSuccess) return e;
    LaunchCfg L(dim3(a.Hkv, (unsigned)blocks), dim3(32 * C::NW), C::SMEM, st, a.flags);
    return cudaLaunchKernelEx(&L.cfg, split4_kernel<D, WIDE, NQ, CHUNK, TW>, s);
  }
  using C = C4<D, WIDE>;
  s.ml = reinterpret_cast<float2*>(w);
  s.acc = reinterpret_cast<float*>(w + p.off_acc);
  s.ctas = p.ctas;
  s.few = 2 * sm_count();
  static bool configured[64] = {};
  cudaError_t e = allow_shared(split4_kernel<D, WIDE, NQ, CHUNK, 1>, C::SMEM, configured);
  if (e != cudaSuccess) return e;
  LaunchCfg L(dim3(p.ctas), dim3(128), C::SMEM, st, a.flags);
  e = cudaLaunchKernelEx(&L.cfg, split4_kernel<D, WIDE, NQ, CHUNK, 1>, s);
  if (e != cudaSuccess) return e;
  const int mass_blocks = a.mass_out ? (a.max_tiles + 255) / 256 : 0;
  // the merge waits for the split kernel on the device, whatever the caller's flags
  // A CTA per row joins many pieces fastest; more rows than two for each SM have few pieces, and a warp does one, eight times
  // fewer CTAs finding their places. (A row / a warp each, us: D 128, 8 heads each, 32 tiles: 24 segments 12.0 / 13.1, 40 15.6 /
  // 14.4, 128 30.5 / 24.6, 512 100.3 / 76.4; D 64, 4 heads: 64 10.9 / 11.1, 128 17.0 / 14.9, 512 52.3 / 41.8.)
  const bool each = (int64_t)a.B * a.Hq <= 2 * sm_count();
  auto merge = [&](auto* kernel, int joins, int64_t rows) {
    LaunchCfg M(dim3(joins + a.Hkv * mass_blocks, (unsigned)rows), dim3(256), 0, st, a.flags | KVARN_LAUNCH_PDL);
    return cudaLaunchKernelEx(&M.cfg, kernel, s, mass_blocks);
  };
  return each ? merge(merge4_kernel<D, C::ROWS, CHUNK, true>, a.Hq, a.B)
              : merge(merge4_kernel<D, C::ROWS, CHUNK, false>, a.Hkv, blocks);
}

template <int D, bool CHUNK>
cudaError_t launch_dim(const Decode4Plan& p, Split4Args& s, void* ws, cudaStream_t st) {
  if constexpr (!CHUNK) {
    if (s.a.G <= 4) return launch_d4<D, false, 1, false>(p, s, ws, st);
  }
  return s.a.io == KVARN_IO_F32 ? launch_d4<D, true, 2, CHUNK>(p, s, ws, st) : launch_d4<D, true, 1, CHUNK>(p, s, ws, st);
}
template <bool CHUNK>
cudaError_t launch_any(const Decode4Plan& p, Split4Args& s, void* ws, cudaStream_t st) {
  switch (s.a.D) {
    case 64: return launch_dim<64, CHUNK>(p, s, ws, st);
    case 128: return launch_dim<128, CHUNK>(p, s, ws, st);
    default: return launch_dim<256, CHUNK>(p, s, ws, st);
  }
}

// segments: (sequence or row group, KV head) pairs, of max_tiles tiles at most.
void make_plan(int64_t segments, int D, bool wide, int max_tiles, size_t tile_parts, Decode4Plan* p) {
  const int resident = D == 64 ? (wide ? C4<64, true>::CTAS : C4<64, false>::CTAS)
                     : D == 128 ? (wide ? C4<128, true>::CTAS : C4<128, false>::CTAS)
                                : (wide ? C4<256, true>::CTAS : C4<256, false>::CTAS);
  const int64_t slots = (int64_t)sm_count() * resident, work = segments * max_tiles, rows = wide ? 8 : 4;
  p->ctas = (int)(work < slots ? work : slots);  // one wave of resident CTAs
  const size_t pieces = (size_t)(p->ctas + segments);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p->off_acc = up(pieces * rows * sizeof(float2));
  p->off_tile = p->off_acc + up(pieces * rows * D * sizeof(float));
  p->ws_bytes = p->off_tile + up(tile_parts * sizeof(float2));
}

}  // namespace

void decode4_plan(int B, int Hq, int Hkv, int D, int max_tiles, Decode4Plan* p) {
  make_plan((int64_t)B * Hkv, D, Hq / Hkv > 4, max_tiles, (size_t)B * Hkv * max_tiles * kRuns * 8, p);
}

cudaError_t launch_decode4(const Decode4Plan& p, const Decode4Args& a, void* ws, cudaStream_t st) {
  Split4Args s{};
  s.a = a;
  return launch_any<false>(p, s, ws, st);
}

// A few positions of one sequence, eight (position, head) rows of a KV head to a segment.
void chunk4_plan(int C, int Hq, int Hkv, int D, int n_tiles, Decode4Plan* p) {
  make_plan((int64_t)Hkv * (((int64_t)C * (Hq / Hkv) + 7) / 8), D, true, n_tiles, 0, p);
}

cudaError_t launch_chunk4(const Prefill4Args& a, int n_tiles, cudaStream_t st) {
  Decode4Plan p;
  chunk4_plan(a.C, a.Hq, a.Hkv, a.D, n_tiles, &p);
  Split4Args s{};
  s.a = Decode4Args{a.q, a.tiles, a.tile_table, nullptr, nullptr, nullptr, a.out, a.tiles_bytes, a.io, a.C, a.Hq,
                    a.Hkv, a.G, a.D, a.table_stride, a.scale, 0, a.err};
  s.pos0 = a.pos0;
  s.n_tiles = n_tiles;
  return launch_any<true>(p, s, a.ws, st);
}

}  // namespace kvarn
