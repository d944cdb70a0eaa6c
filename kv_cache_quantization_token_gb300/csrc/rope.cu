// rope.cu -- queries and keys of new tokens: RMS norm of each head, rotation by position, and a
// Walsh-Hadamard transform of each head, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;   (a, b) -> (a cos - b sin, a sin + b cos);   y H / sqrt(D)
//
// D / 8 threads hold a row (token, head), eight channels each, as two chunks of four that are partners in the
// rotation, so that a pair never leaves its thread; the sum of squares and the transform's far butterflies meet by
// shuffles. Angles are the same for all heads of a token, so a CTA forms them once for its few tokens and keeps
// them in shared memory.
//
// An angle is position * frequency in units of 2^-64 of a turn: a 64-bit integer product drops whole turns
// exactly, whatever the position, and costs three multiply-adds where an fp64 product and its reduction
// would take GB300's slow fp64 units. The quarter turn nearest to it is taken off before it is rounded to fp32.
#include <stdlib.h>
#include "cache4.cuh"

namespace kvarn {
namespace {

#ifndef RB
#define RB 4
#endif
constexpr int kTokens = 16;  // tokens of a CTA at most

// Two chunks of four consecutive elements of a row of type IO.
template <int IO>
struct Chunks {
  uint2 w[IO == KVARN_IO_F32 ? 4 : 2];
  __device__ __forceinline__ void clear() {
    for (auto& x : w) x = make_uint2(0, 0);
  }
  __device__ __forceinline__ void load(const void* p, int64_t i, int c0, int c1) {
    if constexpr (IO == KVARN_IO_F32) {
      const float* q = reinterpret_cast<const float*>(p) + i;
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(q + 4 * c0);
      *reinterpret_cast<uint4*>(w + 2) = *reinterpret_cast<const uint4*>(q + 4 * c1);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
      w[0] = *reinterpret_cast<const uint2*>(q + 4 * c0);
      w[1] = *reinterpret_cast<const uint2*>(q + 4 * c1);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (IO == KVARN_IO_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float((&w[e / 2].x)[e % 2]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u = (&w[e / 2].x)[e % 2];
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
  __device__ __forceinline__ static void store(void* p, int64_t i, int c0, int c1, const float (&x)[8]) {
    io_st4(p, IO, i + 4 * c0, make_float4(x[0], x[1], x[2], x[3]));
    io_st4(p, IO, i + 4 * c1, make_float4(x[4], x[5], x[6], x[7]));
  }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

template <int D, int IO, bool HALVES>
__global__ void __launch_bounds__(256, RB) norm_rotate_kernel(const RopeArgs a, const __grid_constant__ kvarn_rotary_t rot,
                                                          int tokens) {
  constexpr int L = D / 8, ROWS = 32 / L;  // threads of a row, rows of a warp
  __shared__ __align__(16) float cos_s[kTokens][D / 2], sin_s[kTokens][D / 2];
  const int tid = threadIdx.x, lane = tid & 31, l = tid % L;
  const int R = rot.rotary_dim, far = R / 8;  // chunks between partners
  const bool turned = l < far;
  // This thread's chunks. Partners are `far` apart; where that is a power of two, so are all chunks of the row, and a
  // bit of the channel index is a bit of the thread index, which the transform needs.
  const bool bits = !HALVES || (far & (far - 1)) == 0;
  int c0 = 2 * l, c1 = 2 * l + 1;
  if (HALVES) {
    c0 = bits ? 2 * (l & ~(far - 1)) + (l & (far - 1)) : turned ? l : l + far;
    c1 = c0 + (bits || turned ? far : L - far);
  }
  pdl_trigger();
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)min((int64_t)tokens, a.n_tokens - t0);
  // A warp takes ROWS heads of q, or of k, of a token at a time: item w of a token, of nq + nk.
  const int nq = (a.Hq + ROWS - 1) / ROWS, n = nq + (a.Hkv + ROWS - 1) / ROWS, step = 8 * gridDim.y;
  struct Item {
    int t, w;
  };
  auto settle = [&](Item& i) {
    while (i.w >= n) {
      i.w -= n;
      ++i.t;
    }
  };
  auto load = [&](const Item& i, Chunks<IO>& x) {
    const bool is_q = i.w < nq;
    const int h = (is_q ? i.w : i.w - nq) * ROWS + lane / L;
    if (i.t >= nt || h >= (is_q ? a.Hq : a.Hkv)) x.clear();
    else x.load(is_q ? a.q : a.k, (t0 + i.t) * (is_q ? a.q_stride : a.k_stride) + h * D, c0, c1);
  };
  Item now{0, (int)blockIdx.y * 8 + tid / 32};
  settle(now);
  Item next = now;
  next.w += step;
  settle(next);
  Chunks<IO> cur, ahead;
  load(now, cur);
  load(next, ahead);
  Chunks<IO> wq, wk;
  wq.clear();
  wk.clear();
  if (a.q_weight) wq.load(a.q_weight, 0, c0, c1);
  if (a.k_weight) wk.load(a.k_weight, 0, c0, c1);
  for (int i = tid; i < nt * (R / 2); i += 256) {
    const int pair = i % (R / 2), tt = i / (R / 2);
    const uint64_t angle = (uint64_t)a.positions[rot.axis[pair] * a.n_tokens + t0 + tt] * rot.turn[pair];
    const uint32_t quarter = (uint32_t)((angle + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(angle - ((uint64_t)quarter << 62));  // within an eighth of a turn
    float s, c;
    sincospif((float)(int)(rest >> 30) * 1.16415321826934814453125e-10f, &s, &c);  // 2^-33: half turns
    if (quarter & 1) {
      const float x = s;
      s = c;
      c = -x;
    }
    cos_s[tt][pair] = quarter & 2 ? -c : c;
    sin_s[tt][pair] = quarter & 2 ? -s : s;
  }
  __syncthreads();
  while (now.t < nt) {
    const bool is_q = now.w < nq;
    float y[8];
    float2 (&y2)[4] = *reinterpret_cast<float2(*)[4]>(y);
    cur.get(y);
    if (a.eps >= 0.f) {
      float2 ss = mul2(y2[0], y2[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) ss = __ffma2_rn(y2[e], y2[e], ss);
      float sum = ss.x + ss.y;
#pragma unroll
      for (int m = L / 2; m; m >>= 1) sum += shfl_xor(sum, m);
      const float f = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) y2[e] = mul2(y2[e], make_float2(f, f));
      if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
        float w[8];
        Chunks<IO> wc = wq;
        if (!is_q) wc = wk;
        wc.get(w);
#pragma unroll
        for (int e = 0; e < 4; ++e) y2[e] = mul2(y2[e], make_float2(w[2 * e], w[2 * e + 1]));
      }
    }
    if (turned) {
      const float4 c = *reinterpret_cast<const float4*>(cos_s[now.t] + 4 * l);
      const float4 s = *reinterpret_cast<const float4*>(sin_s[now.t] + 4 * l);
      if constexpr (HALVES) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 c2 = e ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
          const float2 s2 = e ? make_float2(s.z, s.w) : make_float2(s.x, s.y);
          const float2 u = y2[e], v = y2[e + 2], m = mul2(v, make_float2(-s2.x, -s2.y));
          y2[e] = __ffma2_rn(u, c2, m);
          y2[e + 2] = __ffma2_rn(u, s2, mul2(v, c2));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ce = (&c.x)[e], se = (&s.x)[e], x = y[2 * e], z = y[2 * e + 1];
          y[2 * e] = fmaf(x, ce, -z * se);
          y[2 * e + 1] = fmaf(x, se, z * ce);
        }
      }
    }
    int d0 = c0, d1 = c1;
    if (a.hadamard) {
      if (!bits) {  // to chunks in order, through shared memory of the warp's own
        __shared__ __align__(16) float row_s[256 * 8];
        float* mine = row_s + (tid - l) * 8;
        *reinterpret_cast<float4*>(mine + 4 * c0) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(mine + 4 * c1) = make_float4(y[4], y[5], y[6], y[7]);
        __syncwarp();
        d0 = 2 * l;
        d1 = 2 * l + 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = mine[8 * l + e];
        __syncwarp();
      }
#pragma unroll
      for (int m = 1; m < 8; m <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(e & m)) {
            const float x = y[e], z = y[e | m];
            y[e] = x + z;
            y[e | m] = x - z;
          }
#pragma unroll
      for (int m = 1; m < L; m <<= 1) {
        const float sign = l & m ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(sign, y[e], shfl_xor(y[e], m));
      }
      const float f = rsqrtf((float)D);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= f;
    }
    const int h = (is_q ? now.w : now.w - nq) * ROWS + lane / L;
    if (h < (is_q ? a.Hq : a.Hkv))
      Chunks<IO>::store(is_q ? a.q_out : a.k_out, (t0 + now.t) * (is_q ? a.qo_stride : a.ko_stride) + h * D, d0, d1, y);
    cur = ahead;
    now = next;
    next.w += step;
    settle(next);
    load(next, ahead);
  }
}

template <int D>
cudaError_t launch_rope(const RopeArgs& a, const kvarn_rotary_t& rot, cudaStream_t st) {
  constexpr int ROWS = 32 / (D / 8);
  const int blocks = ((a.Hq + ROWS - 1) / ROWS + (a.Hkv + ROWS - 1) / ROWS + 7) / 8;  // CTAs for the rows of a token
  const char* E = getenv("ROPE_TOK");
  int tokens = E ? atoi(E) : 4;
  const int64_t grid = (a.n_tokens + tokens - 1) / tokens;
  const int split = grid * blocks <= 8 * (int64_t)sm_count() ? blocks : 1;
  LaunchCfg L(dim3((unsigned)grid, split), dim3(256), 0, st, a.flags);
  const bool halves = rot.rotary_dim > 0 && rot.pairing == KVARN_PAIRS_HALVES;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&L.cfg, kernel, a, rot, tokens); };
  switch (a.io) {
    case KVARN_IO_F32: return halves ? go(norm_rotate_kernel<D, 0, true>) : go(norm_rotate_kernel<D, 0, false>);
    case KVARN_IO_F16: return halves ? go(norm_rotate_kernel<D, 1, true>) : go(norm_rotate_kernel<D, 1, false>);
    default: return halves ? go(norm_rotate_kernel<D, 2, true>) : go(norm_rotate_kernel<D, 2, false>);
  }
}

}  // namespace

cudaError_t launch_norm_rotate(const RopeArgs& a, const kvarn_rotary_t* rotary, cudaStream_t st) {
  kvarn_rotary_t none{};
  const kvarn_rotary_t& rot = rotary ? *rotary : none;
  switch (a.D) {
    case 64: return launch_rope<64>(a, rot, st);
    case 128: return launch_rope<128>(a, rot, st);
    default: return launch_rope<256>(a, rot, st);
  }
}

}  // namespace kvarn
