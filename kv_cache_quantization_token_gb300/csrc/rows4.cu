// rows4.cu -- rows quantised into 4-bit records as they are written, and read back.
//
//   s = least number of 8 significant bits >= max|x| / 7 over 32 channels,  code = x / s to nearest even
//
// A thread holds sixteen channels of K and the same sixteen of V of one row (token, head), so two threads meet for a
// scale and the D / 16 threads of a row for whether it is poison. Both roundings are decided exactly, without a
// division: 7 s and code * s are exact in fp32, so that a candidate is put right by comparisons (below).
//
// What bounds it: instructions and the latency of row, length and table one after another. 7,100 tokens of 8 heads of 128,
// bf16 (37 MB in and out): writing 9.5 us, reading back 7.8, against 5.5 at the copy rate; a token of each of 32 sequences
// both ways 4.0 (4.7 with rows requested once their places are known). Sixteen channels of K and of V to a thread instead
// of eight brought writing from 13.7 to 9.3 (finding a row's place costs as much as coding eight channels); two or four
// rows to a thread gained nothing. Reading takes two runs of eight channels to a thread, so that a warp's stores cover
// whole sectors (9.8 -> 8.1).
#include "cache4.cuh"

namespace kvarn {
namespace {

// The least s >= amax / 7 of at most 8 significant bits, a multiple of 2^-24, at least 2^-24 (amax <= KVARN_MAX4).
// amax * (1/7) is within 2^-22 of the quotient, so that the number below it of that grid is s, or one or two
// steps short; 7 s has 11 bits.
__device__ __forceinline__ float least_scale(float amax) {
  constexpr float kStep = 5.9604644775390625e-8f;  // 2^-24
  const float t = amax * (1.0f / 7.0f);
  const bool small = t < 7.62939453125e-6f;  // 2^-17: the grid is that of multiples of 2^-24
  float s = small ? floorf(t * 16777216.0f) * kStep : __uint_as_float(__float_as_uint(t) & 0xFFFF0000u);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (7.0f * s < amax) s = small ? s + kStep : __uint_as_float(__float_as_uint(s) + 0x10000u);
  return fmaxf(s, kStep);
}

// Two units of eight channels: x / s to the nearest integer, ties to even, plus 8. Added to 1.5 * 2^23 + 8, a
// quotient leaves the nearest integer in the low bits. What of it is next to a border is decided
//   of a 16-bit x by the correctly rounded quotient (an approximate one put right by its exact remainder): x and the
//     borders have too few bits for another number to round onto one;
//   of an fp32 x by x - n s, which is exact there (s has 8 bits, and a difference of about s / 2 needs no more
//     bits than x) and not below s / 2: hardly ever.
template <int IO>
__device__ __forceinline__ uint32_t units_of(const float (&x)[8], float s) {
  constexpr float kRound = 12582920.f;
  const float inv = __fdividef(1.f, s), half = 0.5f * s;
  const float2 inv2 = make_float2(inv, inv), s2 = make_float2(-s, -s), round2 = make_float2(kRound, kRound);
  uint32_t u[8];
  [[maybe_unused]] float r[8], most = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 x2 = make_float2(x[e], x[e + 1]);
    float2 t;
    if constexpr (IO == KVARN_IO_F32) {
      t = __ffma2_rn(x2, inv2, round2);
      const float2 n = __fadd2_rn(t, make_float2(-kRound, -kRound)), d = __ffma2_rn(n, s2, x2);
      r[e] = d.x;
      r[e + 1] = d.y;
      most = fmaxf(most, fmaxf(fabsf(d.x), fabsf(d.y)));
    } else {
      const float2 q = __fmul2_rn(x2, inv2), d = __ffma2_rn(q, s2, x2);
      t = __fadd2_rn(__ffma2_rn(d, inv2, q), round2);
    }
    u[e] = __float_as_uint(t.x);
    u[e + 1] = __float_as_uint(t.y);
  }
  if (IO == KVARN_IO_F32 && most >= half) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(r[e]) > half || (fabsf(r[e]) == half && (u[e] & 1))) u[e] += r[e] > 0.f ? 1 : -1;
  }
  // The bits of 1.5 * 2^23 lie above bit 21, and above bit 31 once shifted by ten: of the sums only the low halves count.
  auto unit = [](const uint32_t* c) { return (((((c[1] << 4) + c[0]) << 4) + c[2]) << 2) + (c[3] << 14) + ((c[3] >> 2) & 3u); };
  return __byte_perm(unit(u), unit(u + 4), 0x5410);
}

// Bits of the largest magnitude of a thread's eight elements, as an fp32 number's (a NaN's are above an infinity's,
// those above every number's).
template <int IO>
__device__ __forceinline__ unsigned largest(const Eight<IO>& v) {
  if constexpr (IO == KVARN_IO_F32) {
    unsigned m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, (&v.w[e / 4].x)[e % 4] & 0x7FFFFFFFu);
    return m;
  } else {  // two 16-bit patterns at a time
    const uint4 w = v.w[0];
    constexpr unsigned kAbs = 0x7FFF7FFFu;
    const unsigned m2 = __vmaxu2(__vmaxu2(w.x & kAbs, w.y & kAbs), __vmaxu2(w.z & kAbs, w.w & kAbs));
    const unsigned m = max(m2 & 0xFFFFu, m2 >> 16);
    return IO == KVARN_IO_F16 ? __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) : m << 16;
  }
}

__device__ __forceinline__ unsigned group_max(unsigned m) {  // over the two threads of 32 channels
  return max(m, __shfl_xor_sync(0xffffffffu, m, 1));
}

// Row t and head h of sequence blockIdx.y, of the threads that hold it, and where its token lies.
struct Place {
  int64_t row;      // b * T + t
  int t, h;
  bool there;       // a row to be moved
  bool inside;      // its token has a place in the table
  bool good;        // the table's record lies inside the pool
  int r;            // token in the run
  int64_t off;      // of the run's bytes
};

template <int D>
__device__ __forceinline__ Place row_of(const Rows4Args& a) {
  constexpr int L = D / 16;
  Place p{};
  const int b = blockIdx.y, i = blockIdx.x * (256 / L) + threadIdx.x / L;
  p.t = i / a.Hkv;
  p.h = i - p.t * a.Hkv;
  p.row = (int64_t)b * a.T + p.t;
  p.there = p.t < a.T && !(a.counts && p.t >= a.counts[b]);
  return p;
}
template <int D>
__device__ __forceinline__ void find(const Rows4Args& a, int first, Place& p) {  // of a row that is there
  const int b = blockIdx.y;
  const int64_t tok = (int64_t)first + p.t;
  p.inside = first >= 0 && tok < (int64_t)kTile * a.max_tiles;
  if (!p.inside) return;
  const int tile = (int)(tok / kTile);
  const int64_t off = a.tile_table[((int64_t)b * a.Hkv + p.h) * a.max_tiles + tile];
  p.good = !(off & 15) && off >= 0 && off <= a.tiles_bytes - Run4<D>::kRecord;
  p.r = (int)tok % kRun;
  p.off = off + (int)tok % kTile / kRun * Run4<D>::kBytes;
}

template <int D, int IO>
__global__ void __launch_bounds__(256) write4_kernel(const Rows4Args a) {
  using R = Run4<D>;
  constexpr int L = D / 16;  // threads of a row
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, c = 16 * (threadIdx.x % L);
  const int first = a.first[blockIdx.y];
  Place p = row_of<D>(a);
  Eight<IO> ek[2]{}, ev[2]{};
  if (p.there) {  // (requested before the row's place is known)
    const int64_t at_k = p.row * a.k_stride + (int64_t)p.h * D + c, at_v = p.row * a.v_stride + (int64_t)p.h * D + c;
    ek[0].load(a.k, at_k);
    ek[1].load(a.k, at_k + 8);
    ev[0].load(a.v, at_v);
    ev[1].load(a.v, at_v + 8);
    find<D>(a, first, p);
    if (c == 0) {
      if (!p.inside) report(a.err, KVARN_DEVERR_WINDOW);
      else if (!p.good) report(a.err, KVARN_DEVERR_RECORD);
    }
  }
  const bool move = p.there && p.inside && p.good;
  const unsigned mk = group_max(max(largest<IO>(ek[0]), largest<IO>(ek[1])));
  const unsigned mv = group_max(max(largest<IO>(ev[0]), largest<IO>(ev[1])));
  const unsigned bad = __ballot_sync(0xffffffffu, max(mk, mv) > __float_as_uint(KVARN_MAX4));
  const bool poison = ((bad >> (lane & ~(L - 1))) & ((1u << L) - 1u)) != 0;
  if (!move) return;
  const float sk = least_scale(__uint_as_float(mk)), sv = least_scale(__uint_as_float(mv));
  auto units = [&](const Eight<IO> (&e)[2], float s) {
    float x[8], y[8];
    e[0].get(x);
    e[1].get(y);
    const uint2 w = make_uint2(units_of<IO>(x, s), units_of<IO>(y, s));
    return poison ? make_uint2(0x22222222u, 0x22222222u) : w;  // (a poisoned token's codes are 0)
  };
  uint8_t* run = a.tiles + p.off;
  *reinterpret_cast<uint2*>(run + R::kKCodes + (c / R::kWide) * (kRun * R::kWide / 2) + p.r * (R::kWide / 2) +
                            c % R::kWide / 2) = units(ek, sk);
  *reinterpret_cast<uint2*>(run + R::kVCodes + (c / 32) * (kRun * 16) + p.r * 16 + c % 32 / 2) = units(ev, sv);
  if (c % 32 == 0) {
    reinterpret_cast<__half*>(run + R::kKScale)[p.r * R::kGroups + c / 32] =
        poison ? __ushort_as_half(0x7FFF) : __float2half_rn(sk);
    reinterpret_cast<__half*>(run + R::kVScale)[c / 32 * kRun + vscale_place(p.r)] =
        poison ? __ushort_as_half(0) : __float2half_rn(sv);
  }
}

template <int D, int IO>
__global__ void __launch_bounds__(256) read4_kernel(const Rows4Args a, uint32_t base) {
  using R = Run4<D>;
  constexpr int L = D / 16;
  pdl_trigger();
  pdl_wait();
  // eight channels of the row's lower half and eight of its upper, so that a warp's stores cover whole sectors
  const int c0 = 8 * (threadIdx.x % L);
  const int first = a.first[blockIdx.y];
  Place p = row_of<D>(a);
  if (!p.there) return;
  find<D>(a, first, p);
  if (c0 == 0) {
    if (!p.inside) report(a.err, KVARN_DEVERR_WINDOW);
    else if (!p.good) report(a.err, KVARN_DEVERR_RECORD);
  }
  if (!p.inside) return;
  uint32_t wk[2] = {}, wv[2] = {};
  __half sk[2], sv[2];
  const uint8_t* run = a.tiles + (p.good ? p.off : 0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = c0 + i * (D / 2);
    sk[i] = __ushort_as_half(0x7FFF);
    sv[i] = __ushort_as_half(0);
    if (p.good) {
      wk[i] = *reinterpret_cast<const uint32_t*>(run + R::kKCodes + (c / R::kWide) * (kRun * R::kWide / 2) +
                                                 p.r * (R::kWide / 2) + c % R::kWide / 2);
      wv[i] = *reinterpret_cast<const uint32_t*>(run + R::kVCodes + (c / 32) * (kRun * 16) + p.r * 16 + c % 32 / 2);
      sk[i] = reinterpret_cast<const __half*>(run + R::kKScale)[p.r * R::kGroups + c / 32];
      sv[i] = reinterpret_cast<const __half*>(run + R::kVScale)[c / 32 * kRun + vscale_place(p.r)];
    }
  }
  auto out = [&](uint32_t w, __half s, void* dst, int64_t at) {
    const __half2 s2 = __half2half2(s);
    uint32_t x[4];  // (channel j, channel j + 4)
    unit_values(w, s2, minus24(s2), base, x);
    if constexpr (IO == KVARN_IO_F16) {  // the values as they are
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dst) + at) =
          make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                     __byte_perm(x[2], x[3], 0x7632));
    } else {
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(as_half2(x[j]));
        y[j] = f.x;
        y[4 + j] = f.y;
      }
      Eight<IO>::store(dst, at, y);
    }
  };
  const int64_t at_k = p.row * a.k_stride + (int64_t)p.h * D + c0, at_v = p.row * a.v_stride + (int64_t)p.h * D + c0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    out(wk[i], sk[i], a.k_out, at_k + i * (D / 2));
    out(wv[i], __hisnan(sk[i]) ? sk[i] : sv[i], a.v_out, at_v + i * (D / 2));
  }
}

template <int D>
LaunchCfg rows_grid(const Rows4Args& a, cudaStream_t st) {
  const int64_t pairs = (int64_t)a.T * a.Hkv, per = 256 / (D / 16);
  return LaunchCfg(dim3((unsigned)((pairs + per - 1) / per), a.B), dim3(256), 0, st, a.flags);
}
template <int D>
cudaError_t write_rows(const Rows4Args& a, cudaStream_t st) {
  const LaunchCfg& L = rows_grid<D>(a, st);
  switch (a.io) {
    case KVARN_IO_F32: return cudaLaunchKernelEx(&L.cfg, write4_kernel<D, 0>, a);
    case KVARN_IO_F16: return cudaLaunchKernelEx(&L.cfg, write4_kernel<D, 1>, a);
    default: return cudaLaunchKernelEx(&L.cfg, write4_kernel<D, 2>, a);
  }
}
template <int D>
cudaError_t read_rows(const Rows4Args& a, cudaStream_t st) {
  const LaunchCfg& L = rows_grid<D>(a, st);
  switch (a.io) {
    case KVARN_IO_F32: return cudaLaunchKernelEx(&L.cfg, read4_kernel<D, 0>, a, kUnitBase);
    case KVARN_IO_F16: return cudaLaunchKernelEx(&L.cfg, read4_kernel<D, 1>, a, kUnitBase);
    default: return cudaLaunchKernelEx(&L.cfg, read4_kernel<D, 2>, a, kUnitBase);
  }
}

}  // namespace

cudaError_t launch_write4(const Rows4Args& a, cudaStream_t st) {
  return a.D == 64 ? write_rows<64>(a, st) : a.D == 128 ? write_rows<128>(a, st) : write_rows<256>(a, st);
}
cudaError_t launch_read4(const Rows4Args& a, cudaStream_t st) {
  return a.D == 64 ? read_rows<64>(a, st) : a.D == 128 ? read_rows<128>(a, st) : read_rows<256>(a, st);
}

}  // namespace kvarn
