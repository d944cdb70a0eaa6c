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
// A poisoned token has NaN in its K image and zeros in its V image, as in its record; tokens behind the last
// position that the chunk sees count as zeros in V, whatever their bytes, and are hidden in the scores.
#include "attend.cuh"
#include "cache4.cuh"

namespace kvarn {
namespace {

template <int D>
__global__ void __launch_bounds__(256) image4_kernel(const Att8Args s) {
  using P = PC8<D, 1>;
  using R = Run4<D>;
  constexpr int KB = P::KB, SUB = P::SUB;
  __shared__ __align__(16) unsigned char rec[R::kRecord];
  const Prefill8Args& a = s.a;
  const int kvh = blockIdx.y, tid = threadIdx.x, j = blockIdx.x;
  pdl_trigger();
  uint8_t* head = a.ws + (int64_t)kvh * s.p.head_imgs * P::IMG;
  const int64_t off = a.tile_table[(int64_t)kvh * a.table_stride + j];
  const bool good = !(off & 15) && off >= 0 && off <= a.tiles_bytes - R::kRecord;
  if (!good && tid == 0) report(a.err, KVARN_DEVERR_RECORD);
  for (int i = tid; i < R::kRecord / 16; i += 256) {
    // (no record: codes and V scales of zero, K scales of NaN)
    const int at = 16 * i % R::kBytes;
    const uint32_t none = at >= R::kKScale && at < R::kVScale ? 0x7FFF7FFFu : 0u;
    *reinterpret_cast<uint4*>(rec + 16 * i) =
        good ? *reinterpret_cast<const uint4*>(a.tiles + off + 16 * i) : make_uint4(none, none, none, none);
  }
  __syncthreads();
  // 16 channels of a token of K, in order
#pragma unroll 2
  for (int x = tid; x < kTile * D / 16; x += 256) {
    const int piece = x & 3, t = (x >> 2) % kTile, c = 64 * (x / (4 * kTile)) + 16 * piece;
    const unsigned char* run = rec + t / kRun * R::kBytes;
    const int r = t % kRun;
    const uint2 w = *reinterpret_cast<const uint2*>(run + R::kKCodes + (c / R::kWide) * (kRun * R::kWide / 2) +
                                                    r * (R::kWide / 2) + c % R::kWide / 2);
    const __half2 sc = __half2half2(reinterpret_cast<const __half*>(run + R::kKScale)[r * R::kGroups + c / 32]);
    const __half2 tc = minus24(sc);
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t v[4];  // (channel e, channel e + 4)
      unit_values(i ? w.y : w.x, sc, tc, kUnitBase, v);
      h[4 * i] = __byte_perm(v[0], v[1], 0x5410);
      h[4 * i + 1] = __byte_perm(v[2], v[3], 0x5410);
      h[4 * i + 2] = __byte_perm(v[0], v[1], 0x7632);
      h[4 * i + 3] = __byte_perm(v[2], v[3], 0x7632);
    }
    const int row = t % KB;
    if (row & 1) {  // the two 16-byte chunks share a 32-byte sector, swapped in odd rows of the swizzle
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t y = h[e];
        h[e] = h[4 + e];
        h[4 + e] = y;
      }
    }
    st_sector(head + image_index(j * SUB + t / KB) * P::IMG + (sw_off(row, c, KB) & ~31u), h);
  }
  // 16 tokens of four channels of V
  const int64_t seen = a.pos0 + a.C - (int64_t)kTile * j;  // tokens of the tile that any row sees
  for (int x = tid; x < D / 4 * (kTile / 16); x += 256) {
    const int tb = x & 3, u = (x >> 2) % (D / 4), t0 = 64 * (x / D) + 16 * tb, c = 4 * u;
    const unsigned char* run = rec + t0 / kRun * R::kBytes;
    const int r = t0 % kRun;
    uint32_t h[4][8];  // [channel][pair of tokens]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(run + R::kVCodes + (c / 32) * (kRun * 16) + (r + 2 * i) * 16) +
                          c % 32 / 4;
      const uint32_t w = (uint32_t)p[0] | (uint32_t)p[8] << 16;
      uint32_t sw = *reinterpret_cast<const uint32_t*>(run + R::kVScale + (c / 32) * 64 + 2 * vscale_place(r + 2 * i));
      const int t = t0 + 2 * i;
      if (t + 1 >= seen) sw = t < seen ? sw & 0xFFFFu : 0u;
      uint32_t v[4];
      unit_values(w, as_half2(sw), minus24(as_half2(sw)), kUnitBase, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e][i] = v[e];
    }
    uint8_t* img = head + (image_index(j * SUB + t0 / KB) + 2) * P::IMG;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = c + e;
      if (row & 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t y = h[e][i];
          h[e][i] = h[e][4 + i];
          h[e][4 + i] = y;
        }
      }
      st_sector(img + (sw_off(row, t0 % KB, D) & ~31u), h[e]);
    }
  }
}

template <int D, int NP>
cudaError_t launch_p4(const Att8Args& s, cudaStream_t st) {
  image4_kernel<D><<<dim3(s.p.n_tsub / PC8<D, 1>::SUB, s.a.Hkv), 256, 0, st>>>(s);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_attend<D, NP, false>(s, st);
}

// Chunks of few score rows per KV head go to the decode kernels, which need no images but go over the cache once
// for every eight rows ("group").
constexpr int64_t kFewGroups = 64, kFewWork = 1600;
int64_t row_groups(int C, int G) { return ((int64_t)C * G + 7) / 8; }
int64_t few_heads(int Hkv) { return Hkv > 6 ? Hkv : 6; }
bool few_rows(int C, int G, int Hkv, int n_tiles) {
  const int64_t groups = row_groups(C, G);
  return groups <= kFewGroups && (groups * Hkv - 5 * few_heads(Hkv)) * n_tiles <= kFewWork;
}

}  // namespace

// At least what every call of at most C positions over at most n_tiles tiles needs, whichever kernels serve it.
size_t prefill4_ws_bytes(int C, int n_tiles, int Hq, int Hkv, int D) {
  const int64_t heads = few_heads(Hkv), sms = sm_count();
  const int64_t groups = row_groups(C, Hq / Hkv), work = (groups < kFewGroups ? groups : kFewGroups) * Hkv;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  // Decode kernels: eight rows for each of a call's pieces, at most a CTA's share each and one more per segment.
  const int64_t entries = 8 * (4 * sms + work);  // (four CTAs per SM at most)
  const size_t few = up((size_t)entries * sizeof(float2)) + up((size_t)entries * D * sizeof(float));
  if (groups * Hkv <= 5 * heads) return few;  // (few_rows holds for every smaller call)
  // Images: those of this call, and the results of key shares, of which there are only as many as fill the SMs
  // once (128 rows to a CTA), and O's emptied sums, of a CTA's rows each.
  const Plan8 p = plan8(C, n_tiles, 0, Hq, Hkv, D, true, false);
  const int64_t ctas = (int64_t)p.row_blocks * Hkv;
  const size_t rows = 128 * (size_t)sms, sums = 128 * (size_t)(ctas > sms ? ctas : sms);
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
  const bool two = a.io == KVARN_IO_F32;
  switch (a.D) {
    case 64: return two ? launch_p4<64, 2>(s, st) : launch_p4<64, 1>(s, st);
    case 128: return two ? launch_p4<128, 2>(s, st) : launch_p4<128, 1>(s, st);
    default: return two ? launch_p4<256, 2>(s, st) : launch_p4<256, 1>(s, st);
  }
}

}  // namespace kvarn
