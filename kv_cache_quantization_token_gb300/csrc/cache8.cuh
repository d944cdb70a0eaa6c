// cache8.cuh -- what the kernels of the 8-bit cache share: the record's field
// offsets, code conversions, element types of queries and outputs, and the
// launchers kvarn8_abi.cu calls.
#pragma once

#include <cuda_bf16.h>

#include "kvarn_common.cuh"

namespace kvarn {

constexpr int kGrp = 16;              // tokens of a scale entry of a record
constexpr int kGrps = kTile / kGrp;   // scale entries per tensor

// Byte offsets of the 8-bit record fields for head_dim D (kvarn_layout8_t).
template <int D>
struct Rec8 {
  static constexpr int kKCodes = 0;                // u8 [16][D/64][8][64]
  static constexpr int kVCodes = kTile * D;        // u8 [D/8][2][8][64]
  static constexpr int kKScale = 2 * kTile * D;    // f32 [8]
  static constexpr int kVScale = kKScale + 4 * kGrps;
  static constexpr int kBytes = kKScale + 128;
};

// Smallest scale of a block: a block of zeros keeps a normal, invertible scale.
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

// Four code bytes (byte i: element i) as two fp16 pairs, exactly: {0, 1} and
// {2, 3}. I8: a byte b beside 0x64 is the fp16 1024 + b, and b = code + 128.
template <int F>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if constexpr (F == KVARN_CODE8_I8) {
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152 = 1024 + 128
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    h01 = *reinterpret_cast<const uint32_t*>(&x);
    h23 = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n"
        " cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(h01), "=r"(h23)
        : "r"(w));
  }
}

// Four consecutive elements of a row of type io (a KVARN_IO_* value known at run time), from i on (a multiple
// of 4, rows 16-byte aligned).
__device__ __forceinline__ float4 io_ld4(const void* p, int io, int64_t i) {
  if (io == KVARN_IO_F32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
  if (io == KVARN_IO_F16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void io_st4(void* p, int io, int64_t i, float4 v) {
  if (io == KVARN_IO_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = v;
  } else if (io == KVARN_IO_F16) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// 2^e that brings a largest magnitude m into [2^top, 2^(top+1)), clamped so that
// it and its inverse are normal; 1 when m is zero, infinite or NaN.
__device__ __forceinline__ float pow2_to(float m, int top) {
  const int ex = (__float_as_int(m) >> 23) & 0xFF;
  int e = (m > 0.f && ex < 255) ? 127 + top - ex : 0;
  e = max(-120, min(120, e));
  return __int_as_float((127 + e) << 23);
}
__device__ __forceinline__ float pow2_inverse(float p) {
  return __int_as_float((254 << 23) - __float_as_int(p));
}

// ---- shared memory, barriers and asynchronous copies ------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive1(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
               : "memory");
}
// Whether the phase of the given parity has completed, without waiting (mbarrier.try_wait may suspend
// the thread).
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait_timed that looks at the clock only after a while: reading the global timer takes longer than
// most waits.
__device__ __forceinline__ bool mbar_wait8(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* stop = nullptr) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (mbar_test_parity(bar, parity)) return true;
  return mbar_wait_timed(bar, parity, err, KVARN_DEVERR_WAIT, stop);
}
// Global -> shared copy (16-byte aligned addresses, size a multiple of 16) that
// completes on bar, whose transaction count was announced by mbar_arrive_tx.
__device__ __forceinline__ void bulk_in(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
// 2^x and log2 x on the special-function unit.
__device__ __forceinline__ float fast_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (x0, x1) as fp16 pairs hi + lo, about 22 significant bits together.
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// ---- launchers -----------------------------------------------------------
cudaError_t launch_compress8(int D, int format, int block_tokens, const float* k_raw,
                             const float* v_raw, int64_t row_stride, int64_t n_rows,
                             const int64_t* src_row0, uint8_t* tiles, int64_t tiles_bytes,
                             const int64_t* dst_record, int64_t n_units, unsigned* err,
                             cudaStream_t st);
cudaError_t launch_expand8(int D, int format, const uint8_t* tiles, int64_t tiles_bytes,
                           const int64_t* src_record, float* k_out, float* v_out,
                           int64_t row_stride, int64_t n_rows, const int64_t* dst_row0,
                           int64_t n_units, unsigned* err, cudaStream_t st);

struct Decode8Plan {
  int span;        // consecutive tiles of a tile item (one CTA)
  int tile_items;  // ceil(max_tiles / span)
  int items;       // tile items + window items
  size_t off_acc;  // workspace offsets: (m, l) per (sequence, head, item) at 0, then the
  size_t off_tile; // accumulators, then (m, l) per (sequence, KV head, tile, head of the group)
  size_t ws_bytes;
};
struct Decode8Args {
  const void* q;
  const uint8_t* tiles;
  const int64_t* tile_table;
  const int32_t* n_tiles;
  const float* win_k;
  const float* win_v;
  const int32_t* win_start;
  const int32_t* win_len;
  const float* mass_in;
  float* mass_out;
  void* out;
  int64_t tiles_bytes;
  int io, win_cap, B, Hq, Hkv, G, D, max_tiles, format;
  float scale;  // softmax scale * log2(e)
  unsigned flags;
  unsigned* err;
};
void decode8_plan(int B, int Hq, int Hkv, int D, int max_tiles, int win_capacity, Decode8Plan* p);
cudaError_t launch_decode8(const Decode8Plan& p, const Decode8Args& a, void* ws, cudaStream_t st);

struct Prefill8Args {
  const void* q;
  const uint8_t* tiles;
  const int64_t* tile_table;  // [Hkv][table_stride]
  const float* win_k;
  const float* win_v;
  uint8_t* ws;
  void* out;
  int64_t pos0, tiles_bytes;
  int io, C, Hq, Hkv, G, D, format, n_tiles, table_stride, win_start, win_len, win_cap;
  float scale;  // softmax scale * log2(e)
  unsigned* err;
};
// Prefill of a few positions by the decode kernels, over the first n_tiles tiles and win_len window rows of a's.
void chunk8_plan(int C, int Hq, int Hkv, int D, int n_tiles, int win_len, Decode8Plan* p);
cudaError_t launch_chunk8(const Prefill8Args& a, int n_tiles, int win_len, cudaStream_t st);
size_t prefill8_ws_bytes(int C, int n_tiles, int win_len, int Hq, int Hkv, int D);
size_t prefill8_ws_bound(int C, int n_tiles, int win_len, int Hq, int Hkv, int D);
cudaError_t launch_prefill8(const Prefill8Args& a, cudaStream_t st);

cudaError_t launch_evict(const int64_t* table, const float* mass, const int32_t* n_tiles,
                         int64_t* table_out, float* mass_out, int32_t* n_out, int64_t* evicted,
                         int B, int Hkv, int max_tiles, int keep, int sinks, int recent,
                         unsigned flags, cudaStream_t st);

}  // namespace kvarn
