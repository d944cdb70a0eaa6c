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
// What bounds it (512 positions, 32 / 8 heads of 128 over 15,500 tokens, bf16: 117 us, 1,095 TFLOP/s, 57%
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
#include "attend.cuh"

namespace kvarn {
namespace {

// ---------------------------------------------------------------------------
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

template <int D, int F, int NP>
cudaError_t launch_p8(const Att8Args& s, cudaStream_t st) {
  using P = PC8<D, NP>;
  const int blocks = s.p.n_tsub / P::SUB + 2 * s.p.n_wsub * (P::KW / kGrp);
  image8_kernel<D, F><<<dim3(blocks, s.a.Hkv), 256, 0, st>>>(s);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_attend<D, NP, true, false>(s, st);
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
  return plan8(C, n_tiles, win_len, Hq, Hkv, D, true, true).bytes;
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
  const Plan8 p = plan8(C, n_tiles, win_len, Hq, Hkv, D, true, true);
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
  s.p = plan8(a.C, n_tblk, win_vis, a.Hq, a.Hkv, a.D, a.io == KVARN_IO_F32, true);
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
