// join.cuh -- what the second kernels of split attention share: the partial results (m, l, acc) of a row's
// items are joined, sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i, and tiles' weights are added up.
// 256 threads per call.
#pragma once

#include "cache8.cuh"

namespace kvarn {

// The items of one row: ml and acc [D] of item i lie at i * STRIDE; the result goes to out as row `row`.
template <int D, int STRIDE = 1>
__device__ __forceinline__ void join_items(const float2* ml, const float* acc, int items, void* out, int io, int64_t row) {
  __shared__ __align__(16) float4 part_s[256];
  __shared__ float2 part_ml[16];
  const int tid = threadIdx.x;
  // each part takes every PARTS-th item of the head with a maximum of its own; the parts meet in shared
  // memory (one round of loads, none waiting for another)
  constexpr int COLS = D / 4, PARTS = 256 / COLS;
  const int col = tid % COLS, pt = tid / COLS;
  float M = -INFINITY, L = 0.f;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = pt; i0 < items; i0 += 4 * PARTS) {
    float2 v[4];
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * PARTS;
      v[k] = i < items ? ml[(int64_t)i * STRIDE] : make_float2(-INFINITY, 0.f);
      x[k] = i < items ? *reinterpret_cast<const float4*>(acc + (int64_t)i * STRIDE * D + 4 * col)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, v[k].x);
    if (m == -INFINITY) continue;  // empty items only
    const float w0 = fast_ex2(M - m);
    L *= w0; sum.x *= w0; sum.y *= w0; sum.z *= w0; sum.w *= w0;
    M = m;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v[k].y != 0.f) {  // an empty item wrote no accumulator
        const float w = fast_ex2(v[k].x - m);
        L = fmaf(w, v[k].y, L);
        sum.x = fmaf(w, x[k].x, sum.x); sum.y = fmaf(w, x[k].y, sum.y);
        sum.z = fmaf(w, x[k].z, sum.z); sum.w = fmaf(w, x[k].w, sum.w);
      }
  }
  part_s[tid] = sum;
  if (col == 0) part_ml[pt] = make_float2(M, L);
  __syncthreads();
  if (tid < COLS) {
    M = -INFINITY;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) M = fmaxf(M, part_ml[p].x);
    L = 0.f;
    sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      const float2 v = part_ml[p];
      if (v.y != 0.f) {
        const float w = fast_ex2(v.x - M);
        const float4 x = part_s[p * COLS + tid];
        L = fmaf(w, v.y, L);
        sum.x = fmaf(w, x.x, sum.x); sum.y = fmaf(w, x.y, sum.y);
        sum.z = fmaf(w, x.z, sum.z); sum.w = fmaf(w, x.w, sum.w);
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    io_st4(out, io, row * D + 4 * tid, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
  }
}

// The same by one warp, for 32 items at most.
template <int D, int STRIDE>
__device__ __forceinline__ void join_few(const float2* ml, const float* acc, int items, void* out, int io, int64_t row) {
  constexpr int N = D < 128 ? 1 : D / 128, PARTS = D < 128 ? 128 / D : 1;  // four channels N times, every PARTS-th item
  const int lane = threadIdx.x & 31, pt = lane % PARTS, col = 4 * (lane / PARTS);
  const float2 v = lane < items ? ml[lane * STRIDE] : make_float2(-INFINITY, 0.f);
  float M = v.x;
  for (int m = 16; m; m >>= 1) M = fmaxf(M, shfl_xor(M, m));
  const float w = v.y != 0.f ? fast_ex2(v.x - M) : 0.f;
  float L = w * v.y;
  for (int m = 16; m; m >>= 1) L += shfl_xor(L, m);
  float4 y[N];
#pragma unroll
  for (int n = 0; n < N; ++n) y[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < items; i0 += 4 * PARTS) {
    float4 x[4][N];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (const int i = i0 + k * PARTS + pt; i < items)
          x[k][n] = *reinterpret_cast<const float4*>(acc + (int64_t)i * STRIDE * D + 128 * n + col);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * PARTS + pt;
      const float f = __shfl_sync(0xffffffffu, w, i & 31);
#pragma unroll
      for (int n = 0; n < N; ++n)
        if (i < items && f != 0.f) {
          y[n].x = fmaf(f, x[k][n].x, y[n].x); y[n].y = fmaf(f, x[k][n].y, y[n].y);
          y[n].z = fmaf(f, x[k][n].z, y[n].z); y[n].w = fmaf(f, x[k][n].w, y[n].w);
        }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int m = 1; m < PARTS; m <<= 1) {
      y[n].x += shfl_xor(y[n].x, m); y[n].y += shfl_xor(y[n].y, m);
      y[n].z += shfl_xor(y[n].z, m); y[n].w += shfl_xor(y[n].w, m);
    }
    if (pt == 0)
      io_st4(out, io, row * D + 128 * n + col, make_float4(y[n].x * inv, y[n].y * inv, y[n].z * inv, y[n].w * inv));
  }
}

// Weights of 256 tiles (from 256 * block on) of one KV head: ml of item i of its query head g at g * head + i * STRIDE,
// tile_ml [tiles][PARTS][8] (maximum, sum) of each tile's parts and heads; n tiles hold tokens, the others keep mass_in.
template <int PARTS, int STRIDE = 1>
__device__ __forceinline__ void join_masses(const float2* ml, int64_t head, int items, const float2* tile_ml, int G, int block, int n,
                                            int max_tiles, const float* mass_in, float* mass_out) {
  __shared__ float2 stat[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = 256 * block + tid;
  // (everything that is read under way together: a tile's parts one after another behind the heads' sums took 4.8 us of
  // a call with four parts and seven heads)
  float2 t[8][PARTS];
  float w = 0.f;
  if (i < max_tiles && mass_in) w = mass_in[i];
#pragma unroll
  for (int h = 0; h < 8; h += 2)
    if (i < n && h < G) {
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        const float4 v = *reinterpret_cast<const float4*>(tile_ml + ((int64_t)i * PARTS + p) * 8 + h);
        t[h][p] = make_float2(v.x, v.y);
        t[h + 1][p] = make_float2(v.z, v.w);
      }
    }
  if (warp < G) {  // (maximum, sum) of query head `warp` of the group
    const float2* row = ml + warp * head;
    float M = -INFINITY, L = 0.f;
    for (int k = lane; k < items; k += 32) M = fmaxf(M, row[(int64_t)k * STRIDE].x);
    for (int m = 16; m; m >>= 1) M = fmaxf(M, shfl_xor(M, m));
    for (int k = lane; k < items; k += 32)
      if (const float2 v = row[(int64_t)k * STRIDE]; v.y != 0.f) L += fast_ex2(v.x - M) * v.y;
    for (int m = 16; m; m >>= 1) L += shfl_xor(L, m);
    if (lane == 0) stat[warp] = make_float2(M, 1.f / L);
  }
  __syncthreads();
  if (i >= max_tiles) return;
  if (i < n) {
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < G) {
#pragma unroll
        for (int p = 0; p < PARTS; ++p) sum += fast_ex2(t[h][p].x - stat[h].x) * t[h][p].y * stat[h].y;
      }
    w += sum;
  }
  mass_out[i] = w;
}

}  // namespace kvarn
