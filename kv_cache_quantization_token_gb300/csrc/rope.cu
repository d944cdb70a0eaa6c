// rope.cu -- queries and keys of new tokens: RMS norm of each head, rotation by position, and a
// Walsh-Hadamard transform of each head, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;   (a, b) -> (a cos - b sin, a sin + b cos);   y H / sqrt(D)
//
// D / 8 threads hold a row (token, head), eight channels each: one 16-byte access per tensor and thread for 16-bit
// rows. Partners of a pair, the sum of squares and the transform's far butterflies meet by shuffles. Angles are the
// same for all heads of a token, so a CTA forms them once for its few tokens, keeps them in shared memory, and a
// thread holds the eight that it needs while it goes over the token's heads.
//
// An angle is position * frequency in units of 2^-64 of a turn: a 64-bit integer product drops whole turns
// exactly, whatever the position, and costs three multiply-adds where an fp64 product and its reduction
// would take GB300's slow fp64 units. The quarter turn nearest to it is taken off before it is rounded to fp32.
#include "cache4.cuh"

namespace kvarn {
namespace {

constexpr int kTokens = 4;  // tokens of a CTA, when there are many

template <int D, int IO>
__global__ void __launch_bounds__(256) norm_rotate_kernel(const RopeArgs a, const __grid_constant__ kvarn_rotary_t rot,
                                                          int tokens, int steps) {
  constexpr int L = D / 8, ROWS = 256 / L;
  __shared__ float2 turn_s[kTokens][D / 2];
  const int tid = threadIdx.x, l = tid % L, H = a.Hq + a.Hkv;
  const int R = rot.rotary_dim, pl = R / 16;
  const bool halves = rot.pairing == KVARN_PAIRS_HALVES;
  pdl_trigger();
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)min((int64_t)tokens, a.n_tokens - t0);
  // step i: heads of token t0 + i / steps
  auto head_of = [&](int i) { return (i % steps * (int)gridDim.y + (int)blockIdx.y) * ROWS + tid / L; };
  auto load = [&](int i, Eight<IO>& x) {
    const int h = head_of(i);
    const int64_t t = t0 + i / steps;
    if (i >= nt * steps || h >= H) {
      for (auto& w : x.w) w = make_uint4(0, 0, 0, 0);
    } else if (h < a.Hq) {
      x.load(a.q, t * a.q_stride + (int64_t)h * D + 8 * l);
    } else {
      x.load(a.k, t * a.k_stride + (int64_t)(h - a.Hq) * D + 8 * l);
    }
  };
  Eight<IO> cur, next;
  load(0, cur);
  Eight<IO> wq{}, wk{};
  if (a.q_weight) wq.load(a.q_weight, 8 * l);
  if (a.k_weight) wk.load(a.k_weight, 8 * l);
  for (int i = tid; i < nt * (R / 2); i += 256) {
    const int pair = i % (R / 2), t = i / (R / 2);
    const uint64_t angle = (uint64_t)a.positions[rot.axis[pair] * a.n_tokens + t0 + t] * rot.turn[pair];
    const uint32_t quarter = (uint32_t)((angle + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(angle - ((uint64_t)quarter << 62));  // within an eighth of a turn
    float s, c;
    sincospif((float)(int)(rest >> 30) * 1.16415321826934814453125e-10f, &s, &c);  // 2^-33: half turns
    if (quarter & 1) {
      const float x = s;
      s = c;
      c = -x;
    }
    if (quarter & 2) {
      s = -s;
      c = -c;
    }
    turn_s[t][pair] = make_float2(c, s);
  }
  __syncthreads();
  float2 cs[8] = {};
  const bool turned = 8 * l < R;
  const int mate = !turned ? l : l < pl ? l + pl : l - pl;
  const float sign = l < pl ? -1.f : 1.f;
  for (int i = 0; i < nt * steps; ++i) {
    load(i + 1, next);
    if (i % steps == 0 && turned) {
      const float2* p = turn_s[i / steps] + (halves ? 8 * (l < pl ? l : l - pl) : 4 * l);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (halves || e < 4) cs[e] = p[e];
    }
    const int h = head_of(i);
    float y[8];
    cur.get(y);
    if (a.eps >= 0.f) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
      for (int m = L / 2; m; m >>= 1) ss += shfl_xor(ss, m);
      const float f = rsqrtf(ss * (1.f / D) + a.eps);
      float w[8];
      if (h < a.Hq) wq.get(w);
      else wk.get(w);
      const bool weighed = h < a.Hq ? a.q_weight != nullptr : a.k_weight != nullptr;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * f * (weighed ? w[e] : 1.f);
    }
    if (R > 0) {
      if (halves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = __shfl_sync(0xffffffffu, y[e], mate, L);
          if (turned) y[e] = fmaf(y[e], cs[e].x, sign * o * cs[e].y);
        }
      } else if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = y[2 * e], z = y[2 * e + 1];
          y[2 * e] = fmaf(x, cs[e].x, -z * cs[e].y);
          y[2 * e + 1] = fmaf(x, cs[e].y, z * cs[e].x);
        }
      }
    }
    if (a.hadamard) {
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
      for (int m = 1; m < L; m <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = shfl_xor(y[e], m);
          y[e] = (l & m) ? o - y[e] : y[e] + o;
        }
      const float f = rsqrtf((float)D);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= f;
    }
    const int64_t t = t0 + i / steps;
    if (h < a.Hq) Eight<IO>::store(a.q_out, t * a.qo_stride + (int64_t)h * D + 8 * l, y);
    else if (h < H) Eight<IO>::store(a.k_out, t * a.ko_stride + (int64_t)(h - a.Hq) * D + 8 * l, y);
    cur = next;
  }
}

template <int D>
cudaError_t launch_rope(const RopeArgs& a, const kvarn_rotary_t& rot, cudaStream_t st) {
  constexpr int ROWS = 256 / (D / 8);
  const int H = a.Hq + a.Hkv, blocks = (H + ROWS - 1) / ROWS;
  // Few tokens: a CTA per row block of a token. Many: kTokens to a CTA, so that their angles keep all of its threads
  // busy and its start is paid once for them.
  const bool many = a.n_tokens >= 8 * kTokens * (int64_t)sm_count();
  const int tokens = many ? kTokens : 1;
  const int64_t grid = (a.n_tokens + tokens - 1) / tokens;
  const int split = grid * blocks <= 8 * (int64_t)sm_count() ? blocks : 1;
  LaunchCfg L(dim3((unsigned)grid, split), dim3(256), 0, st, a.flags);
  const int steps = (blocks + split - 1) / split;
  switch (a.io) {
    case KVARN_IO_F32: return cudaLaunchKernelEx(&L.cfg, norm_rotate_kernel<D, 0>, a, rot, tokens, steps);
    case KVARN_IO_F16: return cudaLaunchKernelEx(&L.cfg, norm_rotate_kernel<D, 1>, a, rot, tokens, steps);
    default: return cudaLaunchKernelEx(&L.cfg, norm_rotate_kernel<D, 2>, a, rot, tokens, steps);
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
