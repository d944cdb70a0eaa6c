// prefill4.cu -- causal attention of a chunk of query positions over 4-bit records: operand images of the cache, and
// the tensor-core kernel over them that the 8-bit cache uses too (attend.cuh).
//
//   out[i][h] = sum_j softmax_j(scale q[i][h] . k_j) v_j over keys j <= pos0 + i
//
//   image kernel   a CTA per tile and KV head: the values, exact in fp16 (code * scale has 11 bits), as operand
//                  images K [key][channel] and V^T [channel][key] of 64-key blocks.
// Since the images hold values, no scales are left for the softmax: a score is a product with the row's scale.
// Precision is that of the 8-bit cache: fp32 queries and weights are fp16 pairs, 16-bit ones one fp16 number.
// Chunks of few rows run on the decode kernels instead (few_rows() below).
//
// What bounds it (512 positions, 32 / 8 heads of 128 over 15,500 tokens, bf16: 104.5 us, 1,224 TFLOP/s, 64% of the measured
// bf16 rate; fp16 111): the products, on the 128 of 152 SMs that have a CTA (tensor pipe 80% busy there), and 13 us of images
// before them. Over the 8-bit cache, with scales in the softmax, it takes 117.
//
// A poisoned token has NaN in its K image and zeros in its V image, as in its record; tokens behind the last
// position that the chunk sees count as zeros in V, whatever their bytes, and are hidden in the scores.
#include "attend.cuh"
#include "cache4.cuh"

namespace kvarn {
namespace {

// Registers x[0..3] of four neighbouring lanes, transposed: lane q of the four gets x[q] of each, in their order.
__device__ __forceinline__ void transpose_quad(uint32_t (&x)[4]) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int m = 1; m < 4; m <<= 1)  // lanes m apart exchange the registers whose index has the other bit
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & m)) {
        const bool high = q & m;
        const uint32_t give = high ? x[i] : x[i | m], got = __shfl_xor_sync(0xffffffffu, give, m);
        x[i] = high ? got : x[i];
        x[i | m] = high ? x[i | m] : got;
      }
}

// Bound by instructions and by writing 64 KB for the 18 that it reads (15,500 tokens, 8 heads of 128: 63 MB to L2 in 13 us;
// with V gathered by 16-bit reads instead of transposed ones 16).
template <int D>
__global__ void __launch_bounds__(256) image4_kernel(const Att8Args s, uint32_t base) {
  using P = PC8<D, 1>;
  using R = Run4<D>;
  constexpr int KB = P::KB, SUB = P::SUB;
  // a tile's V codes and V scales
  constexpr int V_RUN = R::kKScale - R::kVCodes, S_RUN = R::kBytes - R::kVScale;
  __shared__ __align__(16) unsigned char codes[kRuns * V_RUN], scales[kRuns * S_RUN];
  const Prefill8Args& a = s.a;
  const int kvh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j = blockIdx.x;
  pdl_trigger();
  uint8_t* head = a.ws + (int64_t)kvh * s.p.head_imgs * P::IMG;
  const int64_t off = a.tile_table[(int64_t)kvh * a.table_stride + j];
  const bool good = !(off & 15) && off >= 0 && off <= a.tiles_bytes - R::kRecord;
  if (!good && tid == 0) report(a.err, KVARN_DEVERR_RECORD);
  const unsigned char* rec = a.tiles + (good ? off : 0);  // (read only if good; without a record: zero codes, K scales of NaN)
  // K, straight from memory: 16 channels of a token, in order; all loads of V under way before them
  constexpr int NV = kRuns * V_RUN / 16 / 256, NK = kTile * D / 16 / 256;
  uint4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = 16 * (tid + 256 * i);
    v[i] = good ? *reinterpret_cast<const uint4*>(rec + at / V_RUN * R::kBytes + R::kVCodes + at % V_RUN) : make_uint4(0, 0, 0, 0);
  }
  uint4 vs = make_uint4(0, 0, 0, 0);
  const int at_s = 16 * tid;
  if (good && at_s < kRuns * S_RUN)
    vs = *reinterpret_cast<const uint4*>(rec + at_s / S_RUN * R::kBytes + R::kVScale + at_s % S_RUN);
  uint2 kw[NK];
  __half ks[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int x = tid + 256 * i, t = (x >> 2) % kTile, c = 64 * (x / (4 * kTile)) + 16 * (x & 3);
    const unsigned char* run = rec + t / kRun * R::kBytes;
    kw[i] = good ? *reinterpret_cast<const uint2*>(run + R::kKCodes + (c / R::kWide) * (kRun * R::kWide / 2) +
                                                   t % kRun * (R::kWide / 2) + c % R::kWide / 2)
                 : make_uint2(0, 0);
    ks[i] = good ? reinterpret_cast<const __half*>(run + R::kKScale)[t % kRun * R::kGroups + c / 32] : __ushort_as_half(0x7FFF);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) *reinterpret_cast<uint4*>(codes + 16 * (tid + 256 * i)) = v[i];
  if (at_s < kRuns * S_RUN) *reinterpret_cast<uint4*>(scales + at_s) = vs;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int x = tid + 256 * i, t = (x >> 2) % kTile, c = 64 * (x / (4 * kTile)) + 16 * (x & 3);
    const __half2 sc = __half2half2(ks[i]), tc = minus24(sc);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t y[4];  // (channel e, channel e + 4)
      unit_values(k ? kw[i].y : kw[i].x, sc, tc, base, y);
      // (the two 16-byte chunks share a 32-byte sector, swapped in odd rows of the swizzle)
      const int to = (k ^ (t & 1)) ? 4 : 0;
      const uint32_t z[4] = {__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                             __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k == 0) h[e] = h[4 + e] = z[e];
        else if (to) h[4 + e] = z[e];
        else h[e] = z[e];
      }
    }
    st_sector(head + image_index(j * SUB + t / KB) * P::IMG + (sw_off(t % KB, c, KB) & ~31u), h);
  }
  __syncthreads();
  // V, 32 tokens x 32 channels to a warp: read transposed, a lane has two tokens of each eight for four channels; the four
  // lanes of a quad then hold eight tokens of a channel, a chunk of its row, each
  const int64_t seen = a.pos0 + a.C - (int64_t)kTile * j;  // tokens of the tile that any row sees
  const int g = lane >> 2, q = lane & 3;
  for (int x = warp; x < kRuns * (D / 32); x += 8) {
    const int r = x / (D / 32), c = x % (D / 32);
    uint32_t w[4], y[4][4];
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(smem_addr(codes + r * V_RUN + c * 512 + lane * 16))
                 : "memory");
    const uint4 sv = *reinterpret_cast<const uint4*>(scales + r * S_RUN + c * 64 + q * 16);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int t = kRun * r + 8 * m + 2 * q;
      uint32_t sw = (&sv.x)[m];
      if (t + 1 >= seen) sw = t < seen ? sw & 0xFFFFu : 0u;
      uint32_t z[4];
      unit_values(w[m], as_half2(sw), minus24(as_half2(sw)), base, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e][m] = z[e];
    }
    uint8_t* img = head + (image_index(j * SUB + kRun * r / KB) + 2) * P::IMG;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      transpose_quad(y[e]);
      *reinterpret_cast<uint4*>(img + sw_off(32 * c + 4 * g + e, kRun * r % KB + 8 * q, D)) =
          make_uint4(y[e][0], y[e][1], y[e][2], y[e][3]);
    }
  }
}

template <int D, int NP, bool RS>
cudaError_t launch_p4(const Att8Args& s, cudaStream_t st) {
  image4_kernel<D><<<dim3(s.p.n_tsub / PC8<D, 1>::SUB, s.a.Hkv), 256, 0, st>>>(s, kUnitBase);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_attend<D, NP, false, RS>(s, st);
}

template <int D>
cudaError_t launch_p4d(const Att8Args& s, cudaStream_t st) {
  switch (s.a.io) {
    case KVARN_IO_F32: return launch_p4<D, 2, false>(s, st);
    case KVARN_IO_F16: return launch_p4<D, 1, true>(s, st);
    default: return launch_p4<D, 1, false>(s, st);
  }
}

// Chunks of few score rows per KV head go to the decode kernels, which need no images but go over the cache once for
// every eight rows ("group"): some 4.3 ns of all SMs per group and tile of a head (head_dim 128; 2.7 at 64, 7.8 at 256). The images
// with their kernels cost four groups' worth per tile of a head, 24 more per tile, however many heads there are (up to 192
// tiles: a fit), and some 4 us. At head_dim 128, bf16 (us, decode kernels against images):
//   8 KV heads   16 tiles: 6 groups 12.9 / 12.8, 12 15.2 / 13.8;   64: 6 22.3 / 24.1, 8 25.6 / 23.8;   128: 6 33.3 / 31.1;
//                512: 4 73 / 105, 6 106 / 106, 8 137 / 105;   1,024: 4 137 / 198, 8 263 / 198
//   2            64 tiles: 24 22.2 / 23.4, 32 25.7 / 24.2;   128: 16 24.8 / 34.3, 24 33.1 / 27.8;   512: 8 41.0 / 45.7, 24 106 / 44
//   1            128 tiles: 32 24.9 / 33.1, 48 33.3 / 30.4;   512: 16 40.9 / 39.3, 48 106 / 40;   1,024: 8 41 / 50, 32 135 / 53
// Over 2,212 sizes (1 to 16 KV heads, 1 to 64 groups, 4 to 1,024 tiles, each head_dim, fp32 at 128) the choice costs 0.6% on the mean,
// 36% at worst.
constexpr int64_t kFewGroups = 64, kFewWork = 800;
int64_t row_groups(int C, int G) { return ((int64_t)C * G + 7) / 8; }
bool few_rows(int C, int G, int Hkv, int n_tiles) {
  const int64_t groups = row_groups(C, G);
  return groups <= kFewGroups && (groups - 4) * Hkv * n_tiles <= kFewWork + 24 * (n_tiles < 192 ? n_tiles : 192);
}

}  // namespace

// At least what every call of at most C positions over at most n_tiles tiles needs, whichever kernels serve it.
size_t prefill4_ws_bytes(int C, int n_tiles, int Hq, int Hkv, int D) {
  const int64_t sms = sm_count();
  const int64_t groups = row_groups(C, Hq / Hkv), work = (groups < kFewGroups ? groups : kFewGroups) * Hkv;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  // Decode kernels: eight rows for each of a call's pieces, at most a CTA's share each and one more per segment.
  const int64_t entries = 8 * (4 * sms + work);  // (four CTAs per SM at most)
  const size_t few = up((size_t)entries * sizeof(float2)) + up((size_t)entries * D * sizeof(float));
  // (then of every smaller call too: fewer groups only help, and what the tiles' sides differ by is convex in their number)
  if (few_rows(C, Hq / Hkv, Hkv, n_tiles)) return few;
  // Images: those of this call, and the results of key shares, of which there are only as many as fill the SMs
  // once, or kRounds times (128 rows to a CTA), and O's emptied sums, of a CTA's rows each.
  const Plan8 p = plan8(C, n_tiles, 0, Hq, Hkv, D, true, false);
  const int64_t ctas = (int64_t)p.row_blocks * Hkv;
  const int64_t shared = 2 * ctas > sms && p.n_tsub > kShareFrom ? kRounds * sms : sms;
  const size_t rows = 128 * (size_t)shared, sums = 128 * (size_t)(ctas > shared ? ctas : shared);
  const size_t images = p.off_ml + up(rows * sizeof(float2)) + up(rows * D * sizeof(float)) + up(sums * D * sizeof(float));
  return few > images ? few : images;
}

cudaError_t launch_prefill4(const Prefill4Args& a, cudaStream_t st) {
  const int n_tblk = (a.pos0 + a.C - 1) / kTile + 1;  // tiles that the last position sees
  if (few_rows(a.C, a.G, a.Hkv, n_tblk)) return launch_chunk4(a, n_tblk, st);
  Att8Args s{};
  s.a = Prefill8Args{a.q, a.tiles, a.tile_table, nullptr, nullptr, a.ws, a.out, a.pos0, a.tiles_bytes, a.io, a.C, a.Hq,
                     a.Hkv, a.G, a.D, 0, n_tblk, a.table_stride, 0, 0, 0, a.scale, a.err};
  s.p = plan8(a.C, n_tblk, 0, a.Hq, a.Hkv, a.D, a.io == KVARN_IO_F32, false);
  s.ml = reinterpret_cast<float2*>(a.ws + s.p.off_ml);
  s.acc = reinterpret_cast<float*>(a.ws + s.p.off_acc);
  s.sum = reinterpret_cast<float4*>(a.ws + s.p.off_sum);
  switch (a.D) {
    case 64: return launch_p4d<64>(s, st);
    case 128: return launch_p4d<128>(s, st);
    default: return launch_p4d<256>(s, st);
  }
}

}  // namespace kvarn
