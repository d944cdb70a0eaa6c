// decode4.cu -- single-token attention over 4-bit records.
//
//   split kernel   grid (item, KV head, sequence): a CTA of four warps owns `span` consecutive tiles of one KV head, its
//                  warp w the run w (32 tokens) of each. A warp streams its runs by bulk copies of its own and keeps
//                  a softmax of its own; the four meet once, at the item's end, and the item's maximum m, sum l and
//                  accumulator (in units of 2^m) go to the workspace.
//   merge kernel   joins the items of a head, and, on request, adds up each tile's weight.
//
// The warps need no exchange while they run because a run's scores and values both stay in one warp: the codes
// become fp16 numbers in registers, exactly (unit_values), as the A operand of mma.sync m16n8k16, for the scores
// (16 tokens x 16 channels) and, read transposed, for the values (16 channels x 16 tokens). The other operand's eight
// columns are four query heads, each as a pair hi + lo of fp16 (22 bits) in neighbouring columns, so that a lane
// adds the parts of its own accumulators and no product is spent on padding. More than four heads to a group take two
// such sets (NS), which share the unpacked codes. A probability's two parts, in one register, are
// turned into the second product's operand by one movmatrix.
//   s_t = (q . k_t) scale,   O = O 2^(M_old - M) + sum_t 2^(s_t - M) v_t, the sum of a run in accumulators of its own
// (the tensor core drops what falls below a sum's last bit), joined to O with rounding.
//
// The same kernels serve chunks of a few positions (CHUNK): eight (position, head) rows to a CTA, each of which
// sees the cache up to its own position.
#include "cache4.cuh"
#include "join.cuh"

namespace kvarn {
namespace {

constexpr float kNone = -3.0e38f;  // reference exponent before the first run
constexpr float kHead = 14.f;      // probabilities reach 2^14: lo parts stay normal fp16 numbers

template <int D_, int NS_>
struct C4 {
  static constexpr int D = D_, NS = NS_;
  static constexpr int NW = kRuns;             // warps, one per run of a tile
  static constexpr int STG = D == 64 ? 4 : D == 128 ? 3 : NS == 2 ? 3 : 2;  // runs of a warp under way or in use
  static constexpr int CTAS = D == 64 ? (NS == 2 ? 5 : 6) : D == 128 ? 4 : NS == 2 ? 2 : 3;  // resident per SM
  static constexpr int RB = Run4<D>::kBytes;
  static constexpr int OS = D + 8;             // floats of a head's row where the warps meet
  static constexpr int OFF_ML = NW * STG * RB; // float2 [NW][8]: (m, l)
  static constexpr int OFF_BAR = OFF_ML + NW * 64;
  static constexpr int OFF_FLG = OFF_BAR + 8 * NW * STG;
  static constexpr int SMEM = (OFF_FLG + 8 + 127) / 128 * 128;
  static_assert(4 * NS * OS * 4 <= STG * RB, "a warp's accumulators fit in its ring");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit elements, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void load_transposed(const void* p, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(smem_addr(p))
               : "memory");
}

struct Split4Args {
  Decode4Args a;
  float2* ml;       // [rows][items]
  float* acc;       // [rows][items][D]
  float2* tile_ml;  // [B][Hkv][max_tiles][4][8], or NULL
  int span, items;
  int pos0, n_tiles;  // CHUNK: B positions of one sequence instead of B sequences
};

// Score row r (0..7) of a CTA: with CHUNK the (position, head) pairs of a KV head, eight per CTA, are rows of one sequence
// that see the cache up to their own position; otherwise the G heads of sequence blockIdx.z.
struct Row4 {
  bool valid;
  int64_t index;  // among the rows of queries and outputs
  int seen;       // cached tokens that the row sees
};
template <bool CHUNK>
__device__ __forceinline__ Row4 row4(const Split4Args& s, int kvh, int r) {
  const Decode4Args& a = s.a;
  if constexpr (CHUNK) {
    const int64_t n = 8LL * blockIdx.z + r, i = n / a.G;
    const bool valid = i < a.B;
    return Row4{valid, valid ? i * a.Hq + (int64_t)kvh * a.G + n % a.G : 0, valid ? s.pos0 + (int)i + 1 : 0};
  } else {
    return Row4{r < a.G, (int64_t)blockIdx.z * a.Hq + (int64_t)kvh * a.G + min(r, a.G - 1), INT32_MAX};
  }
}

template <int D, int NS, bool CHUNK>
__global__ void __launch_bounds__(128, C4<D, NS>::CTAS) split4_kernel(const Split4Args s) {
  using C = C4<D, NS>;
  using R = Run4<D>;
  constexpr int STG = C::STG, RB = C::RB;
  constexpr int BLK = D / R::kWide;        // blocks of K units
  constexpr int WPB = R::kWide / 32;       // words (8 channels) of a token that a lane holds, per block
  extern __shared__ __align__(128) unsigned char smem[];
  const Decode4Args& a = s.a;
  const int item = blockIdx.x, kvh = blockIdx.y, b = CHUNK ? 0 : blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * STG;
  volatile int* flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLG);
  unsigned char* ring = smem + warp * STG * RB;
  pdl_wait();
  const int first = item * s.span;  // (the last item may own fewer tiles)
  const int stop = min(CHUNK ? s.n_tiles : a.max_tiles, first + s.span);
  const int64_t* table = a.tile_table + ((int64_t)b * a.Hkv + kvh) * a.max_tiles + first;
  // the table's entries of 32 tiles, one per lane, read beside the length
  int64_t entry = first + lane < stop ? table[lane] : 0;
  int len;  // cached tokens that any row of the CTA sees
  if constexpr (CHUNK) {
    len = s.pos0 + min(a.B, (8 * (int)blockIdx.z + 7) / a.G + 1);
  } else {
    len = min(max(a.lens[b], 0), kTile * a.max_tiles);
  }
  const int run0 = kTile * first + kRun * warp;  // first token of this warp
  const int nt = min(max((len - kTile * first + kTile - 1) / kTile, 0), stop - first);
  if (nt <= 0) {
    pdl_trigger();
    if (tid < 4 * NS) {
      const Row4 r = row4<CHUNK>(s, kvh, tid);
      if (r.valid) s.ml[r.index * s.items + item] = make_float2(-INFINITY, 0.f);
    }
    return;
  }
  const int nr = min(nt, max((len - run0 + kTile - 1) / kTile, 0));  // runs of this warp that hold tokens
  if (tid == 0) *flag = 0;
  if (lane == 0) {
    for (int i = 0; i < STG; ++i) mbar_init_n(bar + i, 1);
    mbar_fence_init();
  }
  __syncwarp();
  unsigned bad = 0;  // bit i: the run in slot i has no record
  auto request = [&](int j) {
    if (j >= nr) return;
    const int64_t off = __shfl_sync(0xffffffffu, entry, j & 31);
    const int sl = j % STG;
    bad &= ~(1u << sl);
    if ((off & 15) || off < 0 || off > a.tiles_bytes - R::kRecord) {
      bad |= 1u << sl;
      if (lane == 0) {
        report(a.err, KVARN_DEVERR_RECORD);
        mbar_arrive1(bar + sl);
      }
    } else if (lane == 0) {
      mbar_arrive_tx(bar + sl, RB);
      bulk_in(ring + sl * RB, a.tiles + off + warp * RB, RB, bar + sl);
    }
  };
#pragma unroll
  for (int j = 0; j < STG; ++j) request(j);
  pdl_trigger();

  // B fragments of the query: column g is part g % 2 (hi, lo) of row 4 set + g / 2; a product's channels are those
  // that a word of K units gives to two registers
  uint32_t qb[NS][BLK * WPB][4];
  float c1[NS];             // of the row whose scores this lane holds: row 4 set + q
  [[maybe_unused]] int seen[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const Row4 me = row4<CHUNK>(s, kvh, 4 * n + (g >> 1));
    float x[BLK * WPB][8];
    float mx = 0.f;
#pragma unroll
    for (int w = 0; w < BLK * WPB; ++w) {
      const int c = w / WPB * R::kWide + q * (R::kWide / 4) + 8 * (w % WPB);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 v = me.valid ? io_ld4(a.q, a.io, me.index * D + c + 4 * h) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[w][4 * h] = v.x; x[w][4 * h + 1] = v.y; x[w][4 * h + 2] = v.z; x[w][4 * h + 3] = v.w;
        mx = fmaxf(fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
      }
    }
    mx = fmaxf(mx, shfl_xor(mx, 1));
    mx = fmaxf(mx, shfl_xor(mx, 2));
    const float p2 = pow2_to(mx, 10);
#pragma unroll
    for (int w = 0; w < BLK * WPB; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t hi, lo;
        split_pair(x[w][j] * p2, x[w][j + 4] * p2, hi, lo);
        qb[n][w][j] = (g & 1) ? lo : hi;
      }
    c1[n] = __shfl_sync(0xffffffffu, a.scale * pow2_inverse(p2), 8 * q);
    if constexpr (CHUNK) seen[n] = row4<CHUNK>(s, kvh, 4 * n + q).seen;
  }

  float M[NS], l[NS];
  float o[NS][D / 16][2];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    M[n] = kNone;
    l[n] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = 0.f;
  }
  bool ok = true;
  for (int j = 0; j < nr; ++j) {
    const int sl = j % STG;
    const bool none = bad >> sl & 1;
    const unsigned char* run = ring + sl * RB;
    const int tok0 = run0 + kTile * j;            // position of the run's first token
    const int n_tok = min(kRun, len - tok0);      // tokens of it that are cached
    ok &= mbar_wait8(bar + sl, (uint32_t)(j / STG) & 1u, a.err);
    // scores of tokens 8 x + g of the run, x = 0..3, for row 4 n + q
    float sc[NS][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float e[NS][2][4] = {};  // sums of their own for every other product
#pragma unroll
      for (int k = 0; k < BLK; ++k) {
        uint32_t kw[2][WPB];
        __half2 ks[2], kt[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int t = 16 * mt + 8 * r + g;
          const unsigned char* p = run + R::kKCodes + k * (kRun * R::kWide / 2) + t * (R::kWide / 2) + q * (R::kWide / 8);
          if constexpr (WPB == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            kw[r][0] = v.x; kw[r][1] = v.y; kw[r][2] = v.z; kw[r][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            kw[r][0] = v.x; kw[r][1] = v.y;
          }
          ks[r] = __half2half2(
              reinterpret_cast<const __half*>(run + R::kKScale)[t * R::kGroups + (WPB == 4 ? 4 * k + q : q >> 1)]);
          kt[r] = minus24(ks[r]);
        }
#pragma unroll
        for (int w = 0; w < WPB; ++w) {
          uint32_t x[2][4];
          unit_values(kw[0][w], ks[0], kt[0], x[0]);
          unit_values(kw[1][w], ks[1], kt[1], x[1]);
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            const uint32_t (&f)[4] = qb[n][k * WPB + w];
            mma_f16(e[n][0], x[0][0], x[1][0], x[0][1], x[1][1], f[0], f[1]);
            mma_f16(e[n][1], x[0][2], x[1][2], x[0][3], x[1][3], f[2], f[3]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        sc[n][2 * mt] = ((e[n][0][0] + e[n][1][0]) + (e[n][0][1] + e[n][1][1])) * c1[n];
        sc[n][2 * mt + 1] = ((e[n][0][2] + e[n][1][2]) + (e[n][0][3] + e[n][1][3])) * c1[n];
      }
    }
    if (none) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[n][x] = NAN;
    }
    if (CHUNK || n_tok < kRun) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (8 * x + g >= (CHUNK ? seen[n] - tok0 : n_tok)) sc[n][x] = -INFINITY;
    }
    float alpha[NS];
    uint32_t pb[NS][4];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      float m = fmaxf(fmaxf(sc[n][0], sc[n][1]), fmaxf(sc[n][2], sc[n][3]));
      m = fmaxf(m, shfl_xor(m, 4));
      m = fmaxf(m, shfl_xor(m, 8));
      m = fmaxf(m, shfl_xor(m, 16));
      m = fmaxf(m - kHead, M[n]);
      alpha[n] = fast_ex2(M[n] - m);
      M[n] = m;
      float p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) p[x] = fast_ex2(sc[n][x] - m);
      float sum = (p[0] + p[1]) + (p[2] + p[3]);
      l[n] = fmaf(l[n], alpha[n], sum);
#pragma unroll
      for (int x = 0; x < 4; x += 2) {
        uint32_t hi, lo;
        split_pair(p[x], p[x + 1], hi, lo);
        pb[n][x] = transpose8(__byte_perm(hi, lo, 0x5410));
        pb[n][x + 1] = transpose8(__byte_perm(hi, lo, 0x7632));
      }
      if (s.tile_ml) {  // this run's part of its tile's weight
        sum += shfl_xor(sum, 4);
        sum += shfl_xor(sum, 8);
        sum += shfl_xor(sum, 16);
        if (g == 0)
          s.tile_ml[((((int64_t)b * a.Hkv + kvh) * a.max_tiles + first + j) * kRuns + warp) * 8 + 4 * n + q] =
              make_float2(m, sum);
      }
    }
    if (none) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[n][i][0] *= alpha[n];
          o[n][i][1] *= alpha[n];
        }
    } else {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[4];
        load_transposed(run + R::kVCodes + c * 512 + lane * 16, v);
        uint4 vs = *reinterpret_cast<const uint4*>(run + R::kVScale + c * 64 + q * 16);
        if (n_tok < kRun) {  // what lies behind the last token counts as zeros, whatever it is
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int t = 8 * x + 2 * q;
            (&vs.x)[x] &= t + 1 < n_tok ? 0xFFFFFFFFu : t < n_tok ? 0x0000FFFFu : 0u;
          }
        }
        uint32_t x[4][4];  // [8 tokens][channel]
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const __half2 vv = as_half2((&vs.x)[t]);
          unit_values(v[t], vv, minus24(vv), x[t]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)  // channels 32 c + 4 g + 2 i and the next, in rows g and g + 8
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            float d[4] = {};
            mma_f16(d, x[0][2 * i], x[0][2 * i + 1], x[1][2 * i], x[1][2 * i + 1], pb[n][0], pb[n][1]);
            mma_f16(d, x[2][2 * i], x[2][2 * i + 1], x[3][2 * i], x[3][2 * i + 1], pb[n][2], pb[n][3]);
            float (&y)[2] = o[n][2 * c + i];
            y[0] = fmaf(y[0], alpha[n], d[0] + d[1]);
            y[1] = fmaf(y[1], alpha[n], d[2] + d[3]);
          }
      }
    }
    __syncwarp();  // the slot is used up
    if (((j + STG) & 31) == 0 && j + STG < nr) entry = first + j + STG + lane < stop ? table[j + STG + lane] : 0;
    request(j + STG);
  }
  if (!ok) {  // a copy whose wait ran out still writes to this CTA's memory: each is given as long again
    *flag = 1;
    for (int j = max(0, nr - STG); j < nr; ++j) mbar_wait8(bar + j % STG, (uint32_t)(j / STG) & 1u, nullptr);
  }
  if (s.tile_ml && g == 0)  // runs of the last tile that hold nothing
    for (int j = nr; j < nt; ++j)
#pragma unroll
      for (int n = 0; n < NS; ++n)
        s.tile_ml[((((int64_t)b * a.Hkv + kvh) * a.max_tiles + first + j) * kRuns + warp) * 8 + 4 * n + q] =
            make_float2(kNone, 0.f);
  // the four warps meet: each leaves its rows in its own ring
  float* mine = reinterpret_cast<float*>(ring);
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  __syncwarp();
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    l[n] += shfl_xor(l[n], 4);
    l[n] += shfl_xor(l[n], 8);
    l[n] += shfl_xor(l[n], 16);
    if (g == 0) ml[warp * 8 + 4 * n + q] = make_float2(nr > 0 ? M[n] : -INFINITY, l[n]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      *reinterpret_cast<float2*>(mine + (4 * n + q) * C::OS + 32 * (i / 2) + 4 * g + 2 * (i % 2)) =
          make_float2(o[n][i][0], o[n][i][1]);
  }
  __syncthreads();
  const bool lost = *flag != 0;
  for (int i = tid; i < 4 * NS * (D / 4); i += 128) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    const Row4 me = row4<CHUNK>(s, kvh, r);
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
      const float f = fast_ex2(v[w].x - m);
      const float4 x = *reinterpret_cast<const float4*>(smem + w * STG * RB + (r * C::OS + c) * 4);
      sum = fmaf(f, v[w].y, sum);
      y.x = fmaf(f, x.x, y.x); y.y = fmaf(f, x.y, y.y); y.z = fmaf(f, x.z, y.z); y.w = fmaf(f, x.w, y.w);
    }
    const int64_t part = me.index * s.items + item;
    *reinterpret_cast<float4*>(s.acc + part * D + c) = y;
    if (c == 0) s.ml[part] = lost ? make_float2(0.f, NAN) : make_float2(m, sum);
  }
}

// Joins the items of row blockIdx.x (below Hq), or adds up the weights of 256 tiles of a KV head.
template <int D>
__global__ void __launch_bounds__(256) merge4_kernel(const Split4Args s, int mass_blocks) {
  const Decode4Args& a = s.a;
  const int b = blockIdx.y;
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x >= a.Hq) {
    const int kvh = ((int)blockIdx.x - a.Hq) / mass_blocks, block = ((int)blockIdx.x - a.Hq) % mass_blocks;
    const int64_t at = ((int64_t)b * a.Hkv + kvh) * a.max_tiles;
    const int n = min((int)(((int64_t)max(a.lens[b], 0) + kTile - 1) / kTile), a.max_tiles);
    join_masses<kRuns>(s.ml + ((int64_t)b * a.Hq + kvh * a.G) * s.items, s.items, s.tile_ml + at * kRuns * 8, a.G, block,
                       n, a.max_tiles, a.mass_in ? a.mass_in + at : nullptr, a.mass_out + at);
    return;
  }
  const int64_t row = (int64_t)b * a.Hq + blockIdx.x;
  join_items<D>(s.ml + row * s.items, s.acc + row * s.items * D, s.items, a.out, a.io, row);
}

template <int D, int NS, bool CHUNK>
cudaError_t launch_d4(const Decode4Plan& p, Split4Args& s, void* ws, cudaStream_t st) {
  using C = C4<D, NS>;
  const Decode4Args& a = s.a;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(split4_kernel<D, NS, CHUNK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  unsigned char* w = static_cast<unsigned char*>(ws);
  s.ml = reinterpret_cast<float2*>(w);
  s.acc = reinterpret_cast<float*>(w + p.off_acc);
  s.tile_ml = a.mass_out ? reinterpret_cast<float2*>(w + p.off_tile) : nullptr;
  s.span = p.span;
  s.items = p.items;
  if (p.items > 0) {
    const int64_t rows = (int64_t)a.B * a.G;
    LaunchCfg L(dim3(p.items, a.Hkv, CHUNK ? (unsigned)((rows + 7) / 8) : a.B), dim3(128), C::SMEM, st, a.flags);
    e = cudaLaunchKernelEx(&L.cfg, split4_kernel<D, NS, CHUNK>, s);
    if (e != cudaSuccess) return e;
  }
  const int mass_blocks = a.mass_out ? (a.max_tiles + 255) / 256 : 0;
  // the merge waits for the split kernel on the device, whatever the caller's flags
  LaunchCfg L(dim3(a.Hq + a.Hkv * mass_blocks, a.B), dim3(256), 0, st, a.flags | KVARN_LAUNCH_PDL);
  return cudaLaunchKernelEx(&L.cfg, merge4_kernel<D>, s, mass_blocks);
}

template <bool CHUNK>
cudaError_t launch_any(const Decode4Plan& p, Split4Args& s, void* ws, cudaStream_t st) {
  const bool two = CHUNK || s.a.G > 4;
  switch (s.a.D) {
    case 64: return two ? launch_d4<64, 2, CHUNK>(p, s, ws, st) : launch_d4<64, CHUNK ? 2 : 1, CHUNK>(p, s, ws, st);
    case 128: return two ? launch_d4<128, 2, CHUNK>(p, s, ws, st) : launch_d4<128, CHUNK ? 2 : 1, CHUNK>(p, s, ws, st);
    default: return two ? launch_d4<256, 2, CHUNK>(p, s, ws, st) : launch_d4<256, CHUNK ? 2 : 1, CHUNK>(p, s, ws, st);
  }
}

// groups: CTAs that read a KV head's records; rows: query rows; seqs: sequences of lengths of their own.
void make_plan(int64_t groups, int64_t rows, int seqs, int D, bool two, int max_tiles, size_t tile_parts, Decode4Plan* p) {
  const int ctas = D == 64 ? (two ? C4<64, 2>::CTAS : C4<64, 1>::CTAS)
                 : D == 128 ? (two ? C4<128, 2>::CTAS : C4<128, 1>::CTAS) : (two ? C4<256, 2>::CTAS : C4<256, 1>::CTAS);
  const int64_t slots = (int64_t)sm_count() * ctas, work = groups * max_tiles;
  // whole waves of resident CTAs, as long as an item has at most 32 tiles; several sequences, whose lengths differ
  // as a rule, take two at least
  int64_t waves = (work + 32 * slots - 1) / (32 * slots);
  if (waves < (seqs > 1 ? 2 : 1)) waves = seqs > 1 ? 2 : 1;
  const int64_t span = (work + waves * slots - 1) / (waves * slots);
  p->span = (int)(span < 1 ? 1 : span);
  p->items = (max_tiles + p->span - 1) / p->span;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p->off_acc = up((size_t)rows * p->items * sizeof(float2));
  p->off_tile = p->off_acc + up((size_t)rows * p->items * D * sizeof(float));
  p->ws_bytes = p->off_tile + up(tile_parts * sizeof(float2));
}

}  // namespace

void decode4_plan(int B, int Hq, int Hkv, int D, int max_tiles, Decode4Plan* p) {
  make_plan((int64_t)B * Hkv, (int64_t)B * Hq, B, D, Hq / Hkv > 4, max_tiles, (size_t)B * Hkv * max_tiles * kRuns * 8, p);
}

cudaError_t launch_decode4(const Decode4Plan& p, const Decode4Args& a, void* ws, cudaStream_t st) {
  Split4Args s{};
  s.a = a;
  return launch_any<false>(p, s, ws, st);
}

// A few positions of one sequence, eight (position, head) rows of a KV head to a CTA.
void chunk4_plan(int C, int Hq, int Hkv, int D, int n_tiles, Decode4Plan* p) {
  make_plan((int64_t)Hkv * (((int64_t)C * (Hq / Hkv) + 7) / 8), (int64_t)C * Hq, 1, D, true, n_tiles, 0, p);
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
