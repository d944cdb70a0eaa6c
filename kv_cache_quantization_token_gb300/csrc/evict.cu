// evict.cu -- whole tiles leave the tile table by accumulated attention weight.
//
// Per KV head: of n > keep tiles, the first `sinks`, the last `recent` and the
// keep - sinks - recent heaviest of those between stay, in their old order. A radix
// selection finds the weight T of the lightest tile that stays and how many tiles of weight
// exactly T do (the lowest indices); a running count then moves each tile to its place.
//
// One CTA per sequence: all its KV heads share n, so n_tiles can be updated in place after a
// barrier, and groups of threads (one per KV head) go through the passes in step. The data is
// a few hundred KB at most, read from L1 after the first pass; latency bounds the call.
#include "cache8.cuh"

namespace kvarn {
namespace {

constexpr int kThreads = 1024;

// Unsigned keys in the order of the weights: -0 as 0, NaN as +infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(isnan(w) ? INFINITY : w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// GT: threads per KV head, a power of two of at least 32.
template <int GT>
__global__ void __launch_bounds__(kThreads) evict_kernel(const int64_t* table, const float* mass,
                                                         const int32_t* n_tiles, int64_t* table_out,
                                                         float* mass_out, int32_t* n_out,
                                                         int64_t* evicted, int Hkv, int max_tiles,
                                                         int keep, int sinks, int recent) {
  constexpr int GROUPS = kThreads / GT, GW = GT / 32;
  __shared__ unsigned hist[GROUPS][256];
  __shared__ unsigned found[GROUPS][2];         // digit prefix, how many are still to take
  __shared__ unsigned count[GROUPS][2][GW];     // per warp: tiles of weight T, tiles that stay
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, gi = tid / GT, gt = tid % GT;
  const int lane = tid & 31, gw = gt >> 5;
  const unsigned below = (1u << lane) - 1u;
  const int n = min(max(n_tiles[b], 0), max_tiles);
  __syncthreads();  // every thread has n
  if (tid == 0) n_out[b] = min(n, keep);
  const int lo = sinks, hi = n - recent, take = keep - sinks - recent;
  for (int h0 = 0; h0 < Hkv; h0 += GROUPS) {
    const bool live = h0 + gi < Hkv;
    const int64_t base = ((int64_t)b * Hkv + (live ? h0 + gi : 0)) * max_tiles;
    const int64_t* tab = table + base;
    const float* wt = mass + base;
    int64_t* tab_o = table_out + base;
    float* wt_o = mass_out + base;
    int64_t* ev = evicted ? evicted + base : nullptr;
    if (n <= keep) {  // the same for all heads of the sequence
      if (live)
        for (int i = gt; i < max_tiles; i += GT) {
          const int64_t t = i < n ? tab[i] : -1;
          const float w = i < n ? wt[i] : 0.f;
          tab_o[i] = t;
          wt_o[i] = w;
          if (ev) ev[i] = -1;
        }
      continue;
    }
    unsigned prefix = 0, rem = (unsigned)take;
    if (take > 0) {
#pragma unroll 1
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = gt; i < 256; i += GT) hist[gi][i] = 0u;
        __syncthreads();
        if (live)
          for (int i = lo + gt; i < hi; i += GT) {
            const uint32_t k = weight_key(wt[i]);
            if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[gi][(k >> shift) & 255u], 1u);
          }
        __syncthreads();
        if (gw == 0) {
          // lane l holds digits 255 - 8 l .. 248 - 8 l: the digit at which the running count reaches rem
          unsigned c[8], sum = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += c[i] = hist[gi][255 - 8 * lane - i];
          unsigned before = sum;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const unsigned o = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += o;
          }
          before -= sum;
          if (before < rem && before + sum >= rem) {
            unsigned left = rem - before;
            int i = 0;
            while (left > c[i]) left -= c[i++];
            found[gi][0] = (prefix << 8) | (unsigned)(255 - 8 * lane - i);
            found[gi][1] = left;
          }
        }
        __syncthreads();
        if (live) {
          prefix = found[gi][0];
          rem = found[gi][1];
        }
      }
    }
    unsigned ties = 0, stay = 0;  // tiles of weight T, and tiles that stay, before this run
    for (int i0 = 0; i0 < n; i0 += GT) {
      const int i = i0 + gt;
      const bool in = live && i < n;
      const int64_t t = in ? tab[i] : 0;
      const float w = in ? wt[i] : 0.f;
      const uint32_t k = weight_key(w);
      const bool mid = in && i >= lo && i < hi;
      const unsigned tie_mask = __ballot_sync(0xffffffffu, mid && take > 0 && k == prefix);
      if (lane == 0) count[gi][0][gw] = __popc(tie_mask);
      __syncthreads();
      unsigned tb = ties + __popc(tie_mask & below), all = 0;
      for (int x = 0; x < GW; ++x) {
        const unsigned v = count[gi][0][x];
        tb += x < gw ? v : 0u;
        all += v;
      }
      ties += all;
      const bool stays = in && (!mid || (take > 0 && (k > prefix || (k == prefix && tb < rem))));
      const unsigned stay_mask = __ballot_sync(0xffffffffu, stays);
      if (lane == 0) count[gi][1][gw] = __popc(stay_mask);
      __syncthreads();  // every tile of the run has been read
      unsigned at = stay + __popc(stay_mask & below);
      all = 0;
      for (int x = 0; x < GW; ++x) {
        const unsigned v = count[gi][1][x];
        at += x < gw ? v : 0u;
        all += v;
      }
      stay += all;
      if (stays) {
        tab_o[at] = t;
        wt_o[at] = w;
      } else if (in && ev) {
        ev[i - at] = t;
      }
    }
    __syncthreads();
    if (live)
      for (int i = gt; i < max_tiles; i += GT) {
        if (i >= keep) {
          tab_o[i] = -1;
          wt_o[i] = 0.f;
        }
        if (ev && i >= n - keep) ev[i] = -1;
      }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_evict(const int64_t* table, const float* mass, const int32_t* n_tiles,
                         int64_t* table_out, float* mass_out, int32_t* n_out, int64_t* evicted,
                         int B, int Hkv, int max_tiles, int keep, int sinks, int recent,
                         unsigned flags, cudaStream_t st) {
  LaunchCfg L(dim3(B), dim3(kThreads), 0, st, flags);
#define KVARN_GO(GT)                                                                               \
  cudaLaunchKernelEx(&L.cfg, evict_kernel<GT>, table, mass, n_tiles, table_out, mass_out, n_out,  \
                     evicted, Hkv, max_tiles, keep, sinks, recent)
  if (Hkv <= 1) return KVARN_GO(1024);
  if (Hkv <= 2) return KVARN_GO(512);
  if (Hkv <= 4) return KVARN_GO(256);
  if (Hkv <= 8) return KVARN_GO(128);
  return KVARN_GO(64);
#undef KVARN_GO
}

}  // namespace kvarn
