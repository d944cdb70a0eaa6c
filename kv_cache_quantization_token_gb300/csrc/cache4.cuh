// cache4.cuh -- what the kernels of the 4-bit cache share: the record's field offsets, units
// and scales, rows of eight elements of any input type, and the launchers kvarn4_abi.cu calls.
#pragma once

#include "cache8.cuh"

namespace kvarn {

constexpr int kRun = 32;             // tokens of a run of a record
constexpr int kRuns = kTile / kRun;
constexpr int kGroup4 = 32;          // channels of a scale

// Byte offsets in a run of a 4-bit record for head_dim D (kvarn_layout4_t).
template <int D>
struct Run4 {
  static constexpr int kWide = D < 128 ? D : 128;  // channels of a block of K units
  static constexpr int kGroups = D / kGroup4;
  static constexpr int kKCodes = 0;                // u16 [D/kWide][32][kWide/4]
  static constexpr int kVCodes = 16 * D;           // u16 [D/32][32][8]
  static constexpr int kKScale = 32 * D;           // f16 [32][D/32]
  static constexpr int kVScale = 34 * D;           // f16 [D/32][32]
  static constexpr int kBytes = 36 * D;
  static constexpr int kRecord = kRuns * kBytes;
};
// Place of a token's V scale in its run: the eight tokens whose values a lane holds as pairs
// lie side by side.
__device__ __forceinline__ int vscale_place(int t) { return 8 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1); }

// Two units of one register (low and high half) under scales s = (of the low unit, of the high
// unit) as four pairs of fp16 values: x[j] = (channel j of the low unit, channel j of the high
// unit). A code + 8 at bits 6..9 beside 0x4C00 is the fp16 number 16 + (code + 8), and
// (24 + code) s - 24 s is code s: both products of the one multiply-add are exact (s has 8 bits, 24 s
// has 10, code s 11) and so is its result. t = -24 s; base is kUnitBase, better known at run time only (a kernel
// argument): mask and base are one instruction then, while two constants take an instruction each (11 of
// 15 operations of a word are integer ones with constants, 7 of 11 without: decode of four 64k sequences, head_dim
// 128, executes a fifth less).
constexpr uint32_t kUnitBase = 0x4C004C00u;
__device__ __forceinline__ void unit_values(uint32_t w, __half2 s, __half2 t, uint32_t base, uint32_t (&x)[4]) {
  constexpr uint32_t kMask = 0x03C003C0u;
  const uint32_t u[4] = {(w & kMask) | base, ((w >> 4) & kMask) | base, ((w << 4) & kMask) | base,
                         (__byte_perm(w, 0u, 0x2301) & kMask) | base};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&u[j]), s, t);
    x[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ __half2 minus24(__half2 s) { return __hmul2(s, __half2half2(__ushort_as_half(0xCE00))); }

// Eight consecutive elements of a row of type IO (KVARN_IO_*), from a 16-byte aligned place on.
template <int IO>
struct Eight {
  uint4 w[IO == KVARN_IO_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (IO == KVARN_IO_F32) {
      const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + i);
      w[0] = q[0];
      w[1] = q[1];
    } else {
      w[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (IO == KVARN_IO_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float((&w[e / 4].x)[e % 4]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u = (&w[0].x)[e];
        if constexpr (IO == KVARN_IO_F16) {
          const float2 f = __half22float2(as_half2(u));
          x[2 * e] = f.x;
          x[2 * e + 1] = f.y;
        } else {
          x[2 * e] = __uint_as_float(u << 16);
          x[2 * e + 1] = __uint_as_float(u & 0xFFFF0000u);
        }
      }
    }
  }
  __device__ __forceinline__ static void store(void* p, int64_t i, const float (&x)[8]) {
    if constexpr (IO == KVARN_IO_F32) {
      float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
      q[0] = make_float4(x[0], x[1], x[2], x[3]);
      q[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (IO == KVARN_IO_F16) {
          const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
          (&v.x)[e] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
          (&v.x)[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = v;
    }
  }
};

// ---- launchers -----------------------------------------------------------
struct Rows4Args {
  const void* k;    // rows read (write) ...
  const void* v;
  void* k_out;      // ... or written (read)
  void* v_out;
  uint8_t* tiles;
  const int64_t* tile_table;
  const int32_t* first;   // token of row (b, 0)
  const int32_t* counts;  // or NULL
  int64_t k_stride, v_stride, tiles_bytes;
  int io, B, T, Hkv, D, max_tiles;
  unsigned flags;
  unsigned* err;
};
cudaError_t launch_write4(const Rows4Args& a, cudaStream_t st);
cudaError_t launch_read4(const Rows4Args& a, cudaStream_t st);

struct Decode4Plan {
  int ctas;        // of the split kernel
  size_t off_acc;  // workspace: (m, l) of each piece's rows at 0, then their accumulators, then (m, l) per
  size_t off_tile; // (sequence, KV head, tile, run, head of the group)
  size_t ws_bytes;
};
struct Decode4Args {
  const void* q;
  const uint8_t* tiles;
  const int64_t* tile_table;
  const int32_t* lens;
  const float* mass_in;
  float* mass_out;
  void* out;
  int64_t tiles_bytes;
  int io, B, Hq, Hkv, G, D, max_tiles;
  float scale;  // softmax scale * log2(e)
  unsigned flags;
  unsigned* err;
};
void decode4_plan(int B, int Hq, int Hkv, int D, int max_tiles, Decode4Plan* p);
cudaError_t launch_decode4(const Decode4Plan& p, const Decode4Args& a, void* ws, cudaStream_t st);

struct Prefill4Args {
  const void* q;
  const uint8_t* tiles;
  const int64_t* tile_table;  // [Hkv][table_stride]
  uint8_t* ws;
  void* out;
  int64_t tiles_bytes;
  int pos0, io, C, Hq, Hkv, G, D, table_stride;
  float scale;  // softmax scale * log2(e)
  unsigned* err;
};
// Prefill of a few positions by the decode kernels.
void chunk4_plan(int C, int Hq, int Hkv, int D, int n_tiles, Decode4Plan* p);
cudaError_t launch_chunk4(const Prefill4Args& a, int n_tiles, cudaStream_t st);
size_t prefill4_ws_bytes(int C, int n_tiles, int Hq, int Hkv, int D);
cudaError_t launch_prefill4(const Prefill4Args& a, cudaStream_t st);

struct RopeArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* q_weight;
  const void* k_weight;
  const int64_t* positions;
  int64_t q_stride, k_stride, qo_stride, ko_stride, n_tokens;
  int io, Hq, Hkv, D, hadamard;
  float eps;
  unsigned flags;
};
cudaError_t launch_norm_rotate(const RopeArgs& a, const kvarn_rotary_t* rotary, cudaStream_t st);

}  // namespace kvarn
