// compress8.cu -- 8-bit tile records from raw rows, and raw rows from records.
//
// Per tile, KV head and tensor (K or V), over blocks of `block` tokens x D channels:
//   s = max(max |x| / qmax, 2^-100),  code = the nearest 8-bit value to x / s,
// with ties to even on the exact quotient; expansion is code * s.
//
// Both kernels move 128 D fp32 values and 128 D bytes per tensor and compute a
// dozen instructions per value, so memory bounds them. One CTA per (unit, tensor):
// a thread holds 16 tokens x 4 channels in registers, every load of the CTA is in
// flight at once, and rows are read and written as 16-byte pieces of whole lines.
#include "cache8.cuh"

namespace kvarn {
namespace {

// Thread -> (16-token group, 4-channel column) of a tile. K: the lanes of a warp
// run along the channels. V: four lanes hold the four groups of a 64-token run, so
// that their 16-byte pieces of a channel's codes are one 64-byte line of the record.
template <int D, bool IS_V>
__device__ __forceinline__ void tile_place(int tid, int& grp, int& col) {
  constexpr int COLS = D / 4;
  if constexpr (IS_V) {
    grp = (tid & 3) + 4 * (tid / (4 * COLS));
    col = (tid >> 2) % COLS;
  } else {
    grp = tid / COLS;
    col = tid % COLS;
  }
}

// The quotient x / s for rounding to a code of at most 8 significant bits: within one
// fp32 step of x / s and on the same side of (or equal to) every midpoint of two codes as
// the exact quotient. y is refined once from the reciprocal (Markstein's correction); a
// y that falls on a short value although the remainder is not zero moves one step off it.
__device__ __noinline__ float quotient(float x, float s, float inv) {
  const float y0 = x * inv;
  const float y = fmaf(fmaf(-y0, s, x), inv, y0);
  const float e = fmaf(-y, s, x);  // sign of (x / s - y), s > 0
  const uint32_t u = __float_as_uint(y);
  if ((u & 0xFFFu) == 0u && e != 0.f && (u << 1) != 0u)
    return __uint_as_float((e > 0.f) == (y > 0.f) ? u + 1u : u - 1u);
  return copysignf(y, x);  // (the correction turns -0 into 0)
}
// The same for four values. x * inv is within two steps of the quotient, and the midpoints end in 12
// zero bits: only a product within three steps of such a value (one in 600) needs the care above.
__device__ __forceinline__ void quotients(const float4& x, float s, float inv, float (&y)[4]) {
  y[0] = x.x * inv; y[1] = x.y * inv; y[2] = x.z * inv; y[3] = x.w * inv;
  bool near = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) near |= ((__float_as_uint(y[i]) + 3u) & 0xFFFu) < 7u;
  if (near) {
    y[0] = quotient(x.x, s, inv); y[1] = quotient(x.y, s, inv);
    y[2] = quotient(x.z, s, inv); y[3] = quotient(x.w, s, inv);
  }
}

template <int F>
__device__ __forceinline__ uint32_t encode4(const float (&y)[4]) {
  if constexpr (F == KVARN_CODE8_I8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // rint(y) + 128 in the low byte: adding 1.5 2^23 rounds to the nearest even integer
      const uint32_t r = __float_as_uint(y[i] + 12582912.0f) + 128u;
      w |= (r & 0xFFu) << (8 * i);
    }
    return w;
  } else {
    uint32_t w;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};\n}\n"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return w;
  }
}

template <int D, int F, bool IS_V>
__device__ __forceinline__ void compress_tensor(const float* __restrict__ src, int64_t row_stride,
                                                unsigned char* __restrict__ rec, int block,
                                                unsigned char* img, unsigned* amax_s) {
  constexpr float kQmax = F == KVARN_CODE8_I8 ? 127.f : 448.f;
  const int tid = threadIdx.x;
  int grp, col;
  tile_place<D, IS_V>(tid, grp, col);
  float4 x[16];
  const float* p = src + (int64_t)(16 * grp) * row_stride + 4 * col;
#pragma unroll
  for (int t = 0; t < 16; ++t) x[t] = __ldcs(reinterpret_cast<const float4*>(p + t * row_stride));
  if (tid < kGrps) amax_s[tid] = 0u;
  // magnitudes compare like their bit patterns, with infinity and NaN on top
  unsigned m = 0u;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    m = max(m, max(__float_as_uint(x[t].x) & 0x7FFFFFFFu, __float_as_uint(x[t].y) & 0x7FFFFFFFu));
    m = max(m, max(__float_as_uint(x[t].z) & 0x7FFFFFFFu, __float_as_uint(x[t].w) & 0x7FFFFFFFu));
  }
#pragma unroll
  for (int d = IS_V ? 4 : 1; d < (IS_V || D > 64 ? 32 : 16); d <<= 1)
    m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  __syncthreads();
  if (IS_V ? (tid & 31) < 4 : (tid & (D > 64 ? 31 : 15)) == 0) atomicMax(&amax_s[grp], m);
  __syncthreads();
  const int g0 = grp & ~(block / 16 - 1);
  unsigned bm = 0u;
  for (int g = g0; g < g0 + block / 16; ++g) bm = max(bm, amax_s[g]);
  const bool finite = bm < 0x7F800000u;
  const float s = finite ? fmaxf(__uint_as_float(bm) / kQmax, kScaleFloor) : __int_as_float(0x7FFFFFFF);
  const float inv = 1.0f / s;
  uint32_t w[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    if (finite) quotients(x[t], s, inv, y);
    w[t] = encode4<F>(y);
  }
  if constexpr (IS_V) {
    // 16 tokens of each of the thread's 4 channels, one 16-byte piece per channel
#pragma unroll
    for (int i0 = 0; i0 < 4; ++i0) {
      const int i = i0 ^ (col & 1);  // neighbouring columns store to different banks
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t a = __byte_perm(w[4 * k], w[4 * k + 1], i | ((4 + i) << 4));
        const uint32_t b = __byte_perm(w[4 * k + 2], w[4 * k + 3], i | ((4 + i) << 4));
        o[k] = __byte_perm(a, b, 0x5410);
      }
      const int c = 4 * col + i;
      *reinterpret_cast<uint4*>(img + (c >> 3) * 1024 + (grp >> 2) * 512 + (c & 7) * 64 + (grp & 3) * 16) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
#pragma unroll
    for (int t = 0; t < 16; ++t)
      *reinterpret_cast<uint32_t*>(img + (2 * grp + (t >> 3)) * (8 * D) + ((4 * col) >> 6) * 512 +
                                   (t & 7) * 64 + ((4 * col) & 63)) = w[t];
  }
  // the image goes out with one bulk copy (async proxy: fence the generic writes first)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  using R = Rec8<D>;
  if (tid == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                     rec + (IS_V ? R::kVCodes : R::kKCodes)),
                 "r"((uint32_t)__cvta_generic_to_shared(img)), "r"(kTile * D)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  if (col == 0) reinterpret_cast<float*>(rec + (IS_V ? R::kVScale : R::kKScale))[grp] = s;
  if (IS_V && tid < 4) reinterpret_cast<uint4*>(rec + R::kVScale + 4 * kGrps)[tid] = make_uint4(0, 0, 0, 0);
  if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

template <int D, int F>
__global__ void __launch_bounds__(2 * D) compress8_kernel(const float* __restrict__ k_raw,
                                                          const float* __restrict__ v_raw,
                                                          int64_t row_stride, int64_t n_rows,
                                                          const int64_t* __restrict__ src_row0,
                                                          uint8_t* __restrict__ tiles, int64_t tiles_bytes,
                                                          const int64_t* __restrict__ dst_record,
                                                          int block, unsigned* err) {
  __shared__ __align__(128) unsigned char img[kTile * D];
  __shared__ unsigned amax_s[kGrps];
  const int64_t u = blockIdx.x >> 1;
  const int64_t row0 = src_row0[u], off = dst_record[u];
  if (row0 < 0 || row0 > n_rows - kTile || (off & 15) || off < 0 || off > tiles_bytes - Rec8<D>::kBytes) {
    if (threadIdx.x == 0) report(err, KVARN_DEVERR_RECORD);
    return;
  }
  if (blockIdx.x & 1)
    compress_tensor<D, F, true>(v_raw + row0 * row_stride, row_stride, tiles + off, block, img, amax_s);
  else
    compress_tensor<D, F, false>(k_raw + row0 * row_stride, row_stride, tiles + off, block, img, amax_s);
}

template <int F>
__device__ __forceinline__ float4 decode4(uint32_t w, float s) {
  uint32_t a, b;
  codes_to_half<F>(w, a, b);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
}

template <int D, int F, bool IS_V>
__device__ __forceinline__ void expand_tensor(const unsigned char* __restrict__ rec, bool good,
                                              float* __restrict__ dst, int64_t row_stride) {
  using R = Rec8<D>;
  int grp, col;
  tile_place<D, IS_V>(threadIdx.x, grp, col);
  float* p = dst + (int64_t)(16 * grp) * row_stride + 4 * col;
  uint32_t w[16];  // codes of token t, channels 4 col ..
  float s = __int_as_float(0x7FFFFFFF);
  if (good) {
    s = reinterpret_cast<const float*>(rec + (IS_V ? R::kVScale : R::kKScale))[grp];
    if constexpr (IS_V) {
      uint4 c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ch = 4 * col + i;
        c[i] = *reinterpret_cast<const uint4*>(rec + R::kVCodes + (ch >> 3) * 1024 + (grp >> 2) * 512 +
                                               (ch & 7) * 64 + (grp & 3) * 16);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t c0 = (&c[0].x)[k], c1 = (&c[1].x)[k], c2 = (&c[2].x)[k], c3 = (&c[3].x)[k];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          w[4 * k + t] = __byte_perm(__byte_perm(c0, c1, t | ((4 + t) << 4)),
                                     __byte_perm(c2, c3, t | ((4 + t) << 4)), 0x5410);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 16; ++t)
        w[t] = *reinterpret_cast<const uint32_t*>(rec + R::kKCodes + (2 * grp + (t >> 3)) * (8 * D) +
                                                  ((4 * col) >> 6) * 512 + (t & 7) * 64 + ((4 * col) & 63));
    }
  } else {
#pragma unroll
    for (int t = 0; t < 16; ++t) w[t] = 0u;
  }
#pragma unroll
  for (int t = 0; t < 16; ++t) *reinterpret_cast<float4*>(p + t * row_stride) = decode4<F>(w[t], s);
}

template <int D, int F>
__global__ void __launch_bounds__(2 * D) expand8_kernel(const uint8_t* __restrict__ tiles, int64_t tiles_bytes,
                                                        const int64_t* __restrict__ src_record,
                                                        float* __restrict__ k_out, float* __restrict__ v_out,
                                                        int64_t row_stride, int64_t n_rows,
                                                        const int64_t* __restrict__ dst_row0, unsigned* err) {
  const int64_t u = blockIdx.x >> 1;
  const int64_t row0 = dst_row0[u], off = src_record[u];
  const bool rows_ok = row0 >= 0 && row0 <= n_rows - kTile;
  const bool good = !(off & 15) && off >= 0 && off <= tiles_bytes - Rec8<D>::kBytes;
  if (threadIdx.x == 0 && !(rows_ok && good)) report(err, KVARN_DEVERR_RECORD);
  if (!rows_ok) return;
  if (blockIdx.x & 1)
    expand_tensor<D, F, true>(tiles + off, good, v_out + row0 * row_stride, row_stride);
  else
    expand_tensor<D, F, false>(tiles + off, good, k_out + row0 * row_stride, row_stride);
}

}  // namespace

cudaError_t launch_compress8(int D, int format, int block_tokens, const float* k_raw,
                             const float* v_raw, int64_t row_stride, int64_t n_rows,
                             const int64_t* src_row0, uint8_t* tiles, int64_t tiles_bytes,
                             const int64_t* dst_record, int64_t n_units, unsigned* err,
                             cudaStream_t st) {
  const unsigned grid = (unsigned)(2 * n_units);
#define KVARN_GO(DD, FF)                                                                              \
  compress8_kernel<DD, FF><<<grid, 2 * DD, 0, st>>>(k_raw, v_raw, row_stride, n_rows, src_row0, tiles, \
                                                    tiles_bytes, dst_record, block_tokens, err)
  const bool e = format == KVARN_CODE8_E4M3;
  switch (D) {
    case 64: e ? KVARN_GO(64, 1) : KVARN_GO(64, 0); break;
    case 128: e ? KVARN_GO(128, 1) : KVARN_GO(128, 0); break;
    case 256: e ? KVARN_GO(256, 1) : KVARN_GO(256, 0); break;
    default: return cudaErrorInvalidValue;
  }
#undef KVARN_GO
  return cudaGetLastError();
}

cudaError_t launch_expand8(int D, int format, const uint8_t* tiles, int64_t tiles_bytes,
                           const int64_t* src_record, float* k_out, float* v_out,
                           int64_t row_stride, int64_t n_rows, const int64_t* dst_row0,
                           int64_t n_units, unsigned* err, cudaStream_t st) {
  const unsigned grid = (unsigned)(2 * n_units);
#define KVARN_GO(DD, FF)                                                                                \
  expand8_kernel<DD, FF><<<grid, 2 * DD, 0, st>>>(tiles, tiles_bytes, src_record, k_out, v_out, row_stride, \
                                                  n_rows, dst_row0, err)
  const bool e = format == KVARN_CODE8_E4M3;
  switch (D) {
    case 64: e ? KVARN_GO(64, 1) : KVARN_GO(64, 0); break;
    case 128: e ? KVARN_GO(128, 1) : KVARN_GO(128, 0); break;
    case 256: e ? KVARN_GO(256, 1) : KVARN_GO(256, 0); break;
    default: return cudaErrorInvalidValue;
  }
#undef KVARN_GO
  return cudaGetLastError();
}

}  // namespace kvarn
