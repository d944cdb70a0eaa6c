// rows4.cu -- rows quantised into 4-bit records as they are written, and read back.
//
//   s = least number of 8 significant bits >= max|x| / 7 over 32 channels,  code = x / s to nearest even
//
// A thread holds eight channels of K and the same eight of V of one row (token, head), so four threads meet for a
// scale and the D / 8 threads of a row for whether it is poison; a warp reads 512 consecutive bytes of 16-bit
// rows. Both roundings are decided exactly, without a division: 7 s and code * s are exact in fp32, so that a
// candidate is put right by comparisons (below).
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

// Two units of eight channels: x / s to the nearest integer, ties to even, plus 8. The sum of x / s (with an approximate
// 1 / s) and 1.5 * 2^23 + 8 holds the nearest integer in its low bits. It can be wrong next to a border, where
// x - n s is exact (s has 8 bits, and a difference of about s / 2 needs no more bits than x) and not below s / 2; ties
// of 16-bit rows are such a case in one warp of five, other rows hardly ever.
__device__ __forceinline__ uint32_t units_of(const float (&x)[8], float s) {
  constexpr float kRound = 12582920.f;
  const float inv = __fdividef(1.f, s), half = 0.5f * s;
  const float2 inv2 = make_float2(inv, inv), s2 = make_float2(-s, -s);
  uint32_t u[8];
  float r[8], most = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 x2 = make_float2(x[e], x[e + 1]);
    const float2 t = __ffma2_rn(x2, inv2, make_float2(kRound, kRound));
    const float2 n = __fadd2_rn(t, make_float2(-kRound, -kRound));
    const float2 d = __ffma2_rn(n, s2, x2);
    u[e] = __float_as_uint(t.x);
    u[e + 1] = __float_as_uint(t.y);
    r[e] = d.x;
    r[e + 1] = d.y;
    most = fmaxf(most, fmaxf(fabsf(d.x), fabsf(d.y)));
  }
  if (most >= half) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(r[e]) > half || (fabsf(r[e]) == half && (u[e] & 1))) u[e] += r[e] > 0.f ? 1 : -1;
  }
  // (the bits above a code's four are constant: of 1.5 * 2^23 none among the low 16)
  auto unit = [](const uint32_t* c) {
    return (c[0] & 15u) << 6 | (c[1] & 15u) << 10 | (c[2] & 15u) << 2 | (c[3] & 3u) << 14 | (c[3] & 15u) >> 2;
  };
  return unit(u) | unit(u + 4) << 16;
}

__device__ __forceinline__ unsigned group_max(unsigned m) {  // over the four threads of 32 channels
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Row (b, t) and head of a thread group, and where its token lies.
struct Place {
  int64_t row;      // b * T + t
  int h;
  bool there;       // a row to be moved
  bool inside;      // its token has a place in the table
  int64_t off;      // of the run's bytes in the pool, if its record lies inside
  bool good;
  int r;            // token in the run
};

template <int D>
__device__ __forceinline__ Place place_of(const Rows4Args& a, int64_t pair) {
  Place p{};
  const int64_t rows = (int64_t)a.B * a.T;
  p.row = pair / a.Hkv;
  p.h = (int)(pair - p.row * a.Hkv);
  p.there = p.row < rows;
  if (!p.there) return p;
  const int b = (int)(p.row / a.T), t = (int)(p.row - (int64_t)b * a.T);
  if (a.counts && t >= a.counts[b]) p.there = false;
  const int first = a.first[b];
  const int64_t tok = (int64_t)first + t, tile = tok / kTile;
  p.inside = first >= 0 && tile < a.max_tiles;
  if (!p.there || !p.inside) return p;
  const int64_t off = a.tile_table[((int64_t)b * a.Hkv + p.h) * a.max_tiles + tile];
  p.good = !(off & 15) && off >= 0 && off <= a.tiles_bytes - Run4<D>::kRecord;
  p.r = (int)(tok % kRun);
  p.off = off + (tok % kTile) / kRun * Run4<D>::kBytes;
  return p;
}

template <int D, int IO>
__global__ void __launch_bounds__(256) write4_kernel(const Rows4Args a) {
  using R = Run4<D>;
  constexpr int L = D / 8;  // threads of a row
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, c = 8 * (threadIdx.x % L);
  const int64_t pair = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const Place p = place_of<D>(a, pair);
  if (p.there && c == 0) {
    if (!p.inside) report(a.err, KVARN_DEVERR_WINDOW);
    else if (!p.good) report(a.err, KVARN_DEVERR_RECORD);
  }
  const bool move = p.there && p.inside && p.good;
  float k[8] = {}, v[8] = {};
  if (move) {
    Eight<IO> ek, ev;
    ek.load(a.k, p.row * a.k_stride + (int64_t)p.h * D + c);
    ev.load(a.v, p.row * a.v_stride + (int64_t)p.h * D + c);
    ek.get(k);
    ev.get(v);
  }
  unsigned mk = 0, mv = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mk = max(mk, __float_as_uint(k[e]) & 0x7FFFFFFFu);
    mv = max(mv, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
  mk = group_max(mk);
  mv = group_max(mv);
  // (a NaN's bits are above an infinity's, those above every number's)
  const unsigned bad = __ballot_sync(0xffffffffu, max(mk, mv) > __float_as_uint(KVARN_MAX4));
  const bool poison = L == 32 ? bad != 0 : ((bad >> (lane & ~(L - 1))) & ((1u << (L & 31)) - 1u)) != 0;
  if (!move) return;
  const float sk = least_scale(__uint_as_float(poison ? 0u : mk)), sv = least_scale(__uint_as_float(poison ? 0u : mv));
  if (poison) {
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.f;
  }
  uint8_t* run = a.tiles + p.off;
  *reinterpret_cast<uint32_t*>(run + R::kKCodes + (c / R::kWide) * (kRun * R::kWide / 2) + p.r * (R::kWide / 2) +
                               c % R::kWide / 2) = units_of(k, sk);
  *reinterpret_cast<uint32_t*>(run + R::kVCodes + (c / 32) * (kRun * 16) + p.r * 16 + c % 32 / 2) = units_of(v, sv);
  if (c % 32 == 0) {
    reinterpret_cast<__half*>(run + R::kKScale)[p.r * R::kGroups + c / 32] =
        poison ? __ushort_as_half(0x7FFF) : __float2half_rn(sk);
    reinterpret_cast<__half*>(run + R::kVScale)[c / 32 * kRun + vscale_place(p.r)] =
        poison ? __ushort_as_half(0) : __float2half_rn(sv);
  }
}

template <int D, int IO>
__global__ void __launch_bounds__(256) read4_kernel(const Rows4Args a) {
  using R = Run4<D>;
  constexpr int L = D / 8;
  pdl_trigger();
  pdl_wait();
  const int c = 8 * (threadIdx.x % L);
  const int64_t pair = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const Place p = place_of<D>(a, pair);
  if (!p.there) return;
  if (c == 0) {
    if (!p.inside) report(a.err, KVARN_DEVERR_WINDOW);
    else if (!p.good) report(a.err, KVARN_DEVERR_RECORD);
  }
  if (!p.inside) return;
  uint32_t wk = 0, wv = 0;
  __half sk = __ushort_as_half(0x7FFF), sv = __ushort_as_half(0);
  if (p.good) {
    const uint8_t* run = a.tiles + p.off;
    wk = *reinterpret_cast<const uint32_t*>(run + R::kKCodes + (c / R::kWide) * (kRun * R::kWide / 2) +
                                            p.r * (R::kWide / 2) + c % R::kWide / 2);
    wv = *reinterpret_cast<const uint32_t*>(run + R::kVCodes + (c / 32) * (kRun * 16) + p.r * 16 + c % 32 / 2);
    sk = reinterpret_cast<const __half*>(run + R::kKScale)[p.r * R::kGroups + c / 32];
    sv = reinterpret_cast<const __half*>(run + R::kVScale)[c / 32 * kRun + vscale_place(p.r)];
  }
  if (__hisnan(sk)) sv = sk;
  auto out = [&](uint32_t w, __half s, void* dst, int64_t stride) {
    const __half2 s2 = __half2half2(s);
    uint32_t x[4];
    float y[8];
    unit_values(w, s2, minus24(s2), kUnitBase, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(as_half2(x[j]));
      y[j] = f.x;
      y[4 + j] = f.y;
    }
    Eight<IO>::store(dst, p.row * stride + (int64_t)p.h * D + c, y);
  };
  out(wk, sk, a.k_out, a.k_stride);
  out(wv, sv, a.v_out, a.v_stride);
}

template <int D>
cudaError_t launch_rows(bool write, const Rows4Args& a, cudaStream_t st) {
  const int64_t pairs = (int64_t)a.B * a.T * a.Hkv, per = 256 / (D / 8);
  LaunchCfg L(dim3((unsigned)((pairs + per - 1) / per)), dim3(256), 0, st, a.flags);
  switch (a.io) {
    case KVARN_IO_F32: return cudaLaunchKernelEx(&L.cfg, write ? write4_kernel<D, 0> : read4_kernel<D, 0>, a);
    case KVARN_IO_F16: return cudaLaunchKernelEx(&L.cfg, write ? write4_kernel<D, 1> : read4_kernel<D, 1>, a);
    default: return cudaLaunchKernelEx(&L.cfg, write ? write4_kernel<D, 2> : read4_kernel<D, 2>, a);
  }
}
cudaError_t launch_any(bool write, const Rows4Args& a, cudaStream_t st) {
  switch (a.D) {
    case 64: return launch_rows<64>(write, a, st);
    case 128: return launch_rows<128>(write, a, st);
    default: return launch_rows<256>(write, a, st);
  }
}

}  // namespace

cudaError_t launch_write4(const Rows4Args& a, cudaStream_t st) { return launch_any(true, a, st); }
cudaError_t launch_read4(const Rows4Args& a, cudaStream_t st) { return launch_any(false, a, st); }

}  // namespace kvarn
