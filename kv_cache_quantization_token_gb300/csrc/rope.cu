// rope.cu -- queries and keys of new tokens: RMS norm of each head, rotation by position, and a
// Walsh-Hadamard transform of each head, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;   (a, b) -> (a cos - b sin, a sin + b cos);   y H / sqrt(D)
//
// D / 16 threads of a warp hold a row (token, head), sixteen channels each, as two chunks of eight that are partners in the
// rotation, so that a pair never leaves its thread and a thread's eight angles, which all heads of the token share, stay in
// its registers; the sum of squares and the transform's far butterflies meet by shuffles. The launch's warps share out all
// items (rows of a warp) in order, as equally as whole items
// allow, and stay; they need nothing of one another.
//
// An angle is position * frequency in units of 2^-64 of a turn: a 64-bit integer product drops whole turns
// exactly, whatever the position, and costs three multiply-adds where an fp64 product and its reduction
// would take GB300's slow fp64 units. The quarter turn nearest to it is taken off before it is rounded to fp32.
//
// What bounds it: instructions beside memory. 8,192 tokens of 32 + 8 heads of 128, bf16, packed (168 MB): 30.8 us, 5.4
// TB/s (80% of the copy rate). A warp per token that comes and goes took 37.4, and 38.2 with the frequencies read from the
// launch's arguments, which are served one index at a time (1,337 tokens with transform: 6.3, 7.1, 8.4); twenty warps of 96
// registers instead of sixteen of 128 36.4, two items under way instead of three 32.3, four 30.6; angles of a CTA's tokens in shared
// memory 47 to 58.
#include "cache4.cuh"

namespace kvarn {
namespace {

constexpr int kWarps = 8;  // of a CTA
constexpr int kCtas = 2;   // of an SM
constexpr int kAhead = 3;  // items of a warp under way

// Two chunks of eight consecutive elements of a row of type IO.
template <int IO>
struct Chunks {
  Eight<IO> c[2];
  __device__ __forceinline__ void clear() {
    for (auto& e : c)
      for (auto& x : e.w) x = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const char* p, int apart) {
    c[0].load(p, 0);
    c[1].load(p + apart, 0);
  }
  __device__ __forceinline__ void get(float (&x)[2][8]) const {
    c[0].get(x[0]);
    c[1].get(x[1]);
  }
  __device__ __forceinline__ static void store(char* p, int apart, const float (&x)[2][8]) {
    Eight<IO>::store(p, 0, x[0]);
    Eight<IO>::store(p + apart, 0, x[1]);
  }
};

// (cos, sin) of position * turn: the angle in units of 2^-64 of a turn.
__device__ __forceinline__ float2 turned_by(int64_t position, uint64_t turn) {
  const uint64_t angle = (uint64_t)position * turn;
  const uint32_t quarter = (uint32_t)((angle + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(angle - ((uint64_t)quarter << 62));  // within an eighth of a turn
  float s, c;
  sincospif((float)(int)(rest >> 30) * 1.16415321826934814453125e-10f, &s, &c);  // 2^-33: half turns
  if (quarter & 1) {
    const float y = s;
    s = c;
    c = -y;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

template <int D, int IO, bool HALVES>
__global__ void __launch_bounds__(kWarps * 32, kCtas) norm_rotate_kernel(const RopeArgs a, const __grid_constant__ kvarn_rotary_t rot) {
  constexpr int L = D / 16, ROWS = 32 / L;  // threads of a row, rows of a warp
  constexpr int SIZE = IO == KVARN_IO_F32 ? 4 : 2;
  __shared__ __align__(16) float exchange[kWarps][512];
  __shared__ uint64_t turn_s[128];  // (the launch's arguments, at 32 indexes at once, would be read one by one)
  __shared__ int axis_s[128];
  __shared__ __align__(16) float weight_s[2][D];  // of q, of k: the first halves of all chunks, then the second ones
  const int lane = threadIdx.x & 31, l = lane % L;
  float* mine = exchange[threadIdx.x / 32];
  const int R = rot.rotary_dim, far = R / 16;  // chunks between partners
  const bool turned = l < far;
  // This thread's chunks. Partners are `far` apart; where that is a power of two, so are all chunks of the row, and a
  // bit of the channel index is a bit of the thread index, which the transform needs.
  const bool bits = !HALVES || (far & (far - 1)) == 0;
  int c0 = 2 * l, c1 = 2 * l + 1;
  if (HALVES) {
    c0 = bits ? 2 * (l & ~(far - 1)) + (l & (far - 1)) : turned ? l : l + far;
    c1 = c0 + (bits || turned ? far : L - far);
  }
  for (int i = threadIdx.x; i < R / 2; i += 32 * kWarps) {
    turn_s[i] = rot.turn[i];
    axis_s[i] = rot.axis[i];
  }
  pdl_trigger();
  pdl_wait();
  // Items: ROWS heads of q or of k of a token. This warp's share of all tokens' items in order: `left` of them.
  const int nq = (a.Hq + ROWS - 1) / ROWS, n = nq + (a.Hkv + ROWS - 1) / ROWS;
  const int64_t items = a.n_tokens * n, warps = (int64_t)gridDim.x * kWarps, me = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  const int64_t begin = items * me / warps;
  int left = (int)(items * (me + 1) / warps - begin);
  const int row = lane / L, apart = 8 * SIZE * (c1 - c0);
  // Where the next item lies: heads head .. of the heads of q or k of token t, this thread's first chunk at p.
  struct Cursor {
    char* p;
    int64_t t;
    int head, heads;
    bool k;
  };
  auto enter = [&](Cursor& c, const void* q, int64_t q_stride, const void* k, int64_t k_stride) {
    c.heads = c.k ? a.Hkv : a.Hq;
    c.p = const_cast<char*>(static_cast<const char*>(c.k ? k : q)) + c.t * (c.k ? k_stride : q_stride) * SIZE +
          (int64_t)(c.head + row) * (SIZE * D) + 8 * SIZE * c0;
  };
  auto step = [&](Cursor& c, const void* q, int64_t q_stride, const void* k, int64_t k_stride) {  // true: to another lot of heads
    c.p += ROWS * SIZE * D;
    c.head += ROWS;
    if (c.head < c.heads) return false;
    c.head = 0;
    if (c.k || a.Hkv == 0) ++c.t;
    c.k = !c.k && a.Hkv > 0;
    enter(c, q, q_stride, k, k_stride);
    return true;
  };
  Cursor in;
  in.t = begin / n;
  in.head = (int)(begin - in.t * n);
  in.k = in.head >= nq;
  in.head = (in.k ? in.head - nq : in.head) * ROWS;
  Cursor to = in;
  enter(in, a.q, a.q_stride, a.k, a.k_stride);
  enter(to, a.q_out, a.qo_stride, a.k_out, a.ko_stride);
  // Rows are requested kAhead items before they are worked on, the first ones before the angles are formed. (Rows of an item that
  // are not there hold what they held.)
  int to_load = left;
  auto load = [&](Chunks<IO>& v) {
    if (to_load <= 0) return;
    --to_load;
    if (in.head + row < in.heads) v.load(in.p, apart);
    step(in, a.q, a.q_stride, a.k, a.k_stride);
  };
  Chunks<IO> v[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    v[i].clear();
    load(v[i]);
  }
  for (int i = threadIdx.x; i < 2 * (D / 8); i += 32 * kWarps)
    if (const void* w = i < D / 8 ? a.q_weight : a.k_weight) {
      Eight<IO> e;
      float x[8];
      e.load(w, 8 * (i % (D / 8)));
      e.get(x);
      for (int j = 0; j < 8; ++j) weight_s[i / (D / 8)][j / 4 * (D / 2) + 4 * (i % (D / 8)) + j % 4] = x[j];
    }
  __syncthreads();
  if (left == 0) return;
  // angles of this thread's eight pairs, formed by pairs across the warp
  float2 cs[4], sn[4];
  auto angles = [&]() {
    if (R == 0) return;
    for (int i = lane; i < R / 2; i += 32) {
      const float2 x = turned_by(a.positions[axis_s[i] * a.n_tokens + to.t], turn_s[i]);
      mine[i] = x.x;
      mine[128 + i] = x.y;
    }
    __syncwarp();
    if (turned) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float4 c = *reinterpret_cast<const float4*>(mine + 8 * l + 2 * e);
        const float4 s = *reinterpret_cast<const float4*>(mine + 128 + 8 * l + 2 * e);
        cs[e] = make_float2(c.x, c.y); cs[e + 1] = make_float2(c.z, c.w);
        sn[e] = make_float2(s.x, s.y); sn[e + 1] = make_float2(s.z, s.w);
      }
    }
    __syncwarp();
  };
  const float* wt = nullptr;
  bool weighed = false;
  auto weigh = [&]() {
    wt = weight_s[to.k] + 4 * c0;
    weighed = to.k ? a.k_weight != nullptr : a.q_weight != nullptr;
  };
  angles();
  weigh();
  do {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float y[2][8];
      float2 (&y2)[8] = *reinterpret_cast<float2(*)[8]>(y);
      v[i].get(y);
      load(v[i]);
      if (a.eps >= 0.f) {
        float2 ss = __fmul2_rn(y2[0], y2[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) ss = __ffma2_rn(y2[e], y2[e], ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int m = L / 2; m; m >>= 1) sum += shfl_xor(sum, m);
        const float f = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) y2[e] = __fmul2_rn(y2[e], make_float2(f, f));
        if (weighed) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 x = *reinterpret_cast<const float4*>(wt + e / 2 % 2 * (D / 2) + (e < 4 ? 0 : apart / (2 * SIZE)));
            y2[e] = __fmul2_rn(y2[e], make_float2(x.x, x.y));
            y2[e + 1] = __fmul2_rn(y2[e + 1], make_float2(x.z, x.w));
          }
        }
      }
      if (turned) {
        if constexpr (HALVES) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = y2[e], x = y2[e + 4];
            const float2 m = __fmul2_rn(x, sn[e]);
            y2[e] = __ffma2_rn(u, cs[e], make_float2(-m.x, -m.y));
            y2[e + 4] = __ffma2_rn(u, sn[e], __fmul2_rn(x, cs[e]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float ce = e & 1 ? cs[e / 2].y : cs[e / 2].x, se = e & 1 ? sn[e / 2].y : sn[e / 2].x;
            const float2 u = y2[e];
            y2[e] = make_float2(fmaf(u.x, ce, -u.y * se), fmaf(u.x, se, u.y * ce));
          }
        }
      }
      char* p = to.p;
      int then = apart;
      if (a.hadamard) {
        if (!bits) {  // to chunks in order, through shared memory
          float* of = mine + (lane - l) * 16;
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            *reinterpret_cast<float4*>(of + 8 * c0 + e) = make_float4(y[0][e], y[0][e + 1], y[0][e + 2], y[0][e + 3]);
            *reinterpret_cast<float4*>(of + 8 * c1 + e) = make_float4(y[1][e], y[1][e + 1], y[1][e + 2], y[1][e + 3]);
          }
          __syncwarp();
          p += 8 * SIZE * (2 * l - c0);
          then = 8 * SIZE;
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e / 8][e % 8] = of[16 * l + e];
          __syncwarp();
        }
        // within a pair of elements, then pairs at a time
#pragma unroll
        for (int e = 0; e < 8; ++e) y2[e] = make_float2(y2[e].x + y2[e].y, y2[e].x - y2[e].y);
#pragma unroll
        for (int m = 1; m < 8; m <<= 1)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(e & m)) {
              const float2 u = y2[e], x = y2[e | m];
              y2[e] = __fadd2_rn(u, x);
              y2[e | m] = __ffma2_rn(x, make_float2(-1.f, -1.f), u);
            }
#pragma unroll
        for (int m = 1; m < L; m <<= 1) {
          const float sign = l & m ? -1.f : 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y2[e] = __ffma2_rn(make_float2(sign, sign), y2[e], make_float2(shfl_xor(y2[e].x, m), shfl_xor(y2[e].y, m)));
        }
        const float f = rsqrtf((float)D);
#pragma unroll
        for (int e = 0; e < 8; ++e) y2[e] = __fmul2_rn(y2[e], make_float2(f, f));
      }
      if (to.head + row < to.heads) Chunks<IO>::store(p, then, y);
      if (--left == 0) break;
      if (step(to, a.q_out, a.qo_stride, a.k_out, a.ko_stride)) {
        if (!to.k) angles();
        weigh();
      }
    }
  } while (left > 0);
}

template <int D>
cudaError_t launch_rope(const RopeArgs& a, const kvarn_rotary_t& rot, cudaStream_t st) {
  constexpr int ROWS = 32 / (D / 16);
  const int64_t n = (a.Hq + ROWS - 1) / ROWS + (a.Hkv + ROWS - 1) / ROWS;
  const int64_t resident = kCtas * (int64_t)sm_count(), ctas = (a.n_tokens * n + kWarps - 1) / kWarps;
  LaunchCfg L(dim3((unsigned)(ctas < resident ? ctas : resident)), dim3(kWarps * 32), 0, st, a.flags);
  const bool halves = rot.rotary_dim > 0 && rot.pairing == KVARN_PAIRS_HALVES;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&L.cfg, kernel, a, rot); };
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
