// compress8.cu -- 8-bit tile records from raw rows, and raw rows from records.
//
// Per tile, KV head and tensor (K or V), over blocks of `block` tokens x D channels:
//   s = max(max |x| / qmax, 2^-100),  code = the nearest 8-bit value to x / s,
// with ties to even on the exact quotient; expansion is code * s.
//
// Both kernels move 128 D fp32 values and 128 D bytes per tensor and compute some ten
// instructions per value, so memory bounds them. Compression holds 8 tokens x 4 channels in a thread's
// registers, expansion 16 x 4, and rows are read and written as 16-byte pieces of whole lines.
// 335 MB each: compressed in 63 us at head_dim 128 (5.3 TB/s), 63 us at 64 and 68 us at 256, expanded in 54
// to 55 us (6.2 TB/s). With 16 tokens per thread, half the warps, compression took 66, 64 and 71; with
// rows in a ring of half tensors 69, 80 and 75; loading straight into registers 66, 68 and 98.
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
  const float2 i2 = make_float2(inv, inv);
  const float2 a = __fmul2_rn(make_float2(x.x, x.y), i2), b = __fmul2_rn(make_float2(x.z, x.w), i2);
  y[0] = a.x; y[1] = a.y; y[2] = b.x; y[3] = b.y;
  unsigned near = 0xFFFFFFFFu;  // the least (bits + 3) mod 2^12, in the upper 12 bits
#pragma unroll
  for (int i = 0; i < 4; ++i) near = min(near, (__float_as_uint(y[i]) << 20) + (3u << 20));
  if (near < (7u << 20)) {
    y[0] = quotient(x.x, s, inv); y[1] = quotient(x.y, s, inv);
    y[2] = quotient(x.z, s, inv); y[3] = quotient(x.w, s, inv);
  }
}

template <int F>
__device__ __forceinline__ uint32_t encode4(const float (&y)[4]) {
  if constexpr (F == KVARN_CODE8_I8) {
    // adding 1.5 2^23 rounds to the nearest even integer, whose low byte, with its top bit turned
    // over, is the code + 128
    const float2 magic = make_float2(12582912.0f, 12582912.0f);
    const float2 a = __fadd2_rn(make_float2(y[0], y[1]), magic), b = __fadd2_rn(make_float2(y[2], y[3]), magic);
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410) ^ 0x80808080u;
  } else {
    uint32_t w;
    asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};\n}\n"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    return w;
  }
}

// Compression: a CTA goes over (unit, tensor) pairs. The rows of the next one arrive in shared memory by
// bulk copies while the codes of this one, whose rows are in registers, are formed.
template <int D>
struct C8 {
  static constexpr int NTHR = 4 * D;             // 8 tokens x 4 channels each
  static constexpr int IN = kTile * D * 4;       // rows of one tensor
  static constexpr int OFF_IMG = IN;             // its codes
  static constexpr int OFF_BAR = OFF_IMG + kTile * D;
  static constexpr int OFF_AMAX = OFF_BAR + 8;   // unsigned [8]
  static constexpr int OFF_META = OFF_AMAX + 4 * kGrps;  // int64 [2]: record offset, -1 if refused
  static constexpr int SMEM = (OFF_META + 16 + 127) / 128 * 128;
  static constexpr int CTAS = D == 64 ? 4 : D == 128 ? 2 : 1;  // resident per SM: 128 KB of rows under way
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

template <int D, int F>
__global__ void __launch_bounds__(C8<D>::NTHR, C8<D>::CTAS)
compress8_kernel(const float* __restrict__ k_raw, const float* __restrict__ v_raw, int64_t row_stride,
                 int64_t n_rows, const int64_t* __restrict__ src_row0, uint8_t* __restrict__ tiles,
                 int64_t tiles_bytes, const int64_t* __restrict__ dst_record, int64_t n_pairs, int block,
                 unsigned* err) {
  using C = C8<D>;
  using R = Rec8<D>;
  constexpr float kQmax = F == KVARN_CODE8_I8 ? 127.f : 448.f;
  constexpr int COLS = D / 4;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* img = smem + C::OFF_IMG;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  unsigned* amax_s = reinterpret_cast<unsigned*>(smem + C::OFF_AMAX);
  volatile int64_t* meta = reinterpret_cast<volatile int64_t*>(smem + C::OFF_META);
  const int tid = threadIdx.x, lane = tid & 31;
  // the first warp keeps the offsets of the pair after the next in registers
  int64_t row0 = 0, off = 0;
  auto look_up = [&](int64_t x) {
    if (x < n_pairs) {
      row0 = src_row0[x >> 1];
      off = dst_record[x >> 1];
    }
  };
  auto inside = [&](int64_t row, int64_t rec) {
    return row >= 0 && row <= n_rows - kTile && !(rec & 15) && rec >= 0 && rec <= tiles_bytes - R::kBytes;
  };
  // requests the rows of pair x, whose offsets were looked up; one warp
  auto request = [&](int64_t x, int slot) {
    const bool good = inside(row0, off);
    if (lane == 0) {
      meta[slot] = good ? off : -1;
      if (good) mbar_arrive_tx(bar, C::IN);
      else mbar_arrive1(bar);
      if (!good) report(err, KVARN_DEVERR_RECORD);
    }
    __syncwarp();
    if (!good) return;
    const float* src = ((x & 1) ? v_raw : k_raw) + row0 * row_stride;
    if (row_stride == D) {
      if (lane == 0) bulk_in(smem, src, C::IN, bar);
    } else {
      for (int t = lane; t < kTile; t += 32) bulk_in(smem + t * D * 4, src + t * row_stride, D * 4, bar);
    }
  };
  if (tid == 0) {
    mbar_init_n(bar, 1);
    mbar_fence_init();
  }
  __syncthreads();
  if (tid < 32) {
    look_up(blockIdx.x);
    request(blockIdx.x, 0);
    look_up((int64_t)blockIdx.x + gridDim.x);
  }
  __syncthreads();  // (keeps the set-up out of the loop's registers: without it the loop spills, 115 us for 113)
  uint32_t n = 0;
  int64_t x = blockIdx.x;
  for (; x < n_pairs; x += gridDim.x, ++n) {
    const bool is_v = x & 1;
    // group of 8 tokens and column of 4 channels. K: the lanes of a warp run along the channels. V: 8 columns
    // and 4 groups, whose 8-byte pieces of a channel's codes are half a line of the record.
    const int grp = is_v ? ((lane >> 3) + 4 * (tid / (4 * COLS))) : tid / COLS;
    const int col = is_v ? (lane & 7) + 8 * ((tid >> 5) % (COLS / 8)) : tid % COLS;
    const bool landed = mbar_wait8(bar, n & 1u, err);
    float4 r[8];
    const float4* p = reinterpret_cast<const float4*>(smem) + (8 * grp) * COLS + col;
#pragma unroll
    for (int t = 0; t < 8; ++t) r[t] = p[t * COLS];
    const int64_t rec_off = meta[n & 1u];
    if (tid < kGrps) amax_s[tid] = 0u;
    if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the codes before are out
    if (!__syncthreads_and(landed)) break;  // (joined: what follows has barriers)
    if (tid < 32 && x + gridDim.x < n_pairs) {
      request(x + gridDim.x, (n + 1) & 1u);
      look_up(x + 2 * (int64_t)gridDim.x);
    }
    if (rec_off < 0) {
      __syncthreads();
      continue;
    }
    float top = 0.f;
    float2 odd = make_float2(0.f, 0.f);  // 0, or NaN with a NaN or an infinity among the values
    const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      top = fmaxf(fmaxf(top, fabsf(r[t].x)), fabsf(r[t].y));
      top = fmaxf(fmaxf(top, fabsf(r[t].z)), fabsf(r[t].w));
      odd = __ffma2_rn(make_float2(r[t].x, r[t].y), zero, odd);
      odd = __ffma2_rn(make_float2(r[t].z, r[t].w), zero, odd);
    }
    // magnitudes compare like their bit patterns, with infinity and NaN on top
    unsigned m = odd.x + odd.y == 0.f ? __float_as_uint(top) : 0x7F800000u;
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
    if ((lane & 7) == 0) atomicMax(&amax_s[grp >> 1], m);
    __syncthreads();
    const int g0 = (grp >> 1) & ~(block / 16 - 1);
    unsigned bm = 0u;
    for (int g = g0; g < g0 + block / 16; ++g) bm = max(bm, amax_s[g]);
    const bool finite = bm < 0x7F800000u;
    const float s = finite ? fmaxf(__uint_as_float(bm) / kQmax, kScaleFloor) : __int_as_float(0x7FFFFFFF);
    const float inv = 1.0f / s;
    uint32_t w[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      if (finite) quotients(r[t], s, inv, y);
      w[t] = encode4<F>(y);
    }
    if (is_v) {
      // 8 tokens of each of the thread's 4 channels, one 8-byte piece per channel
#pragma unroll
      for (int i0 = 0; i0 < 4; ++i0) {
        const int i = i0 ^ (col & 1);  // neighbouring columns store to different banks
        uint32_t o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t a = __byte_perm(w[4 * k], w[4 * k + 1], i | ((4 + i) << 4));
          const uint32_t b = __byte_perm(w[4 * k + 2], w[4 * k + 3], i | ((4 + i) << 4));
          o[k] = __byte_perm(a, b, 0x5410);
        }
        const int c = 4 * col + i;
        *reinterpret_cast<uint2*>(img + (c >> 3) * 1024 + (grp >> 3) * 512 + (c & 7) * 64 + (grp & 7) * 8) =
            make_uint2(o[0], o[1]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        *reinterpret_cast<uint32_t*>(img + grp * (8 * D) + ((4 * col) >> 6) * 512 + t * 64 + ((4 * col) & 63)) = w[t];
    }
    // the codes go out with one bulk copy (async proxy: fence the generic writes first)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    unsigned char* rec = tiles + rec_off;
    if (tid == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                       rec + (is_v ? R::kVCodes : R::kKCodes)),
                   "r"(smem_addr(img)), "r"(kTile * D)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if (col == 0 && !(grp & 1)) reinterpret_cast<float*>(rec + (is_v ? R::kVScale : R::kKScale))[grp >> 1] = s;
    if (is_v && tid < 4) reinterpret_cast<uint4*>(rec + R::kVScale + 4 * kGrps)[tid] = make_uint4(0, 0, 0, 0);
  }
  if (x < n_pairs) {
    // A wait ran out, for some threads or all, and the CTA has given up as one. The copy under way is given as long
    // again, as it writes to this CTA's memory; this pair's and the following ones' scales are NaN.
    mbar_wait8(bar, n & 1u, nullptr);
    for (; x < n_pairs; x += gridDim.x) {
      const int64_t rec = dst_record[x >> 1];
      if (tid < kGrps && inside(src_row0[x >> 1], rec))
        reinterpret_cast<float*>(tiles + rec + ((x & 1) ? R::kVScale : R::kKScale))[tid] = __int_as_float(0x7FFFFFFF);
    }
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
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

template <int D, int F>
cudaError_t launch_c8(int block, const float* k_raw, const float* v_raw, int64_t row_stride, int64_t n_rows,
                      const int64_t* src_row0, uint8_t* tiles, int64_t tiles_bytes, const int64_t* dst_record,
                      int64_t n_units, unsigned* err, cudaStream_t st) {
  using C = C8<D>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(compress8_kernel<D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int64_t pairs = 2 * n_units, slots = (int64_t)sm_count() * C::CTAS;
  // an even grid: a CTA stays with one tensor
  const unsigned grid = (unsigned)(pairs < slots ? pairs : slots & ~(int64_t)1);
  compress8_kernel<D, F><<<grid, C::NTHR, C::SMEM, st>>>(k_raw, v_raw, row_stride, n_rows, src_row0, tiles,
                                                         tiles_bytes, dst_record, pairs, block, err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compress8(int D, int format, int block_tokens, const float* k_raw,
                             const float* v_raw, int64_t row_stride, int64_t n_rows,
                             const int64_t* src_row0, uint8_t* tiles, int64_t tiles_bytes,
                             const int64_t* dst_record, int64_t n_units, unsigned* err,
                             cudaStream_t st) {
#define KVARN_GO(DD, FF)                                                                          \
  launch_c8<DD, FF>(block_tokens, k_raw, v_raw, row_stride, n_rows, src_row0, tiles, tiles_bytes, \
                    dst_record, n_units, err, st)
  const bool e = format == KVARN_CODE8_E4M3;
  switch (D) {
    case 64: return e ? KVARN_GO(64, 1) : KVARN_GO(64, 0);
    case 128: return e ? KVARN_GO(128, 1) : KVARN_GO(128, 0);
    case 256: return e ? KVARN_GO(256, 1) : KVARN_GO(256, 0);
    default: return cudaErrorInvalidValue;
  }
#undef KVARN_GO
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
