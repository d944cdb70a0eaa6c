// kvarn4_abi.cu -- the extern "C" entry points of the 4-bit cache and of kvarn_norm_rotate: arguments are checked on
// the host, and nothing is enqueued when they are wrong.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "cache4.cuh"

namespace {

bool dim_ok(int D) { return D == 64 || D == 128 || D == 256; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA; }
bool io_ok(int io) { return io == KVARN_IO_F32 || io == KVARN_IO_F16 || io == KVARN_IO_BF16; }
int io_size(int io) { return io == KVARN_IO_F32 ? 4 : 2; }
bool flags_ok(unsigned f) { return !(f & ~KVARN_LAUNCH_PDL); }

// A layout handed back by the caller must be one this library produced.
bool layout_ok(const kvarn_layout4_t* L) {
  kvarn_layout4_t ref;
  return kvarn_layout4(L->head_dim, &ref) == KVARN_OK && memcmp(&ref, L, sizeof(ref)) == 0;
}

int heads_ok(int Hq, int Hkv, int D) {
  if (!dim_ok(D)) return KVARN_ERR_UNSUPPORTED;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hkv > 65535) return KVARN_ERR_BAD_ARG;
  if (Hq / Hkv > 8) return KVARN_ERR_UNSUPPORTED;
  return KVARN_OK;
}

// Token positions stay below 2^31.
constexpr int kMostTiles = (1 << 24) - 1;
// Tiles of all KV heads of a prefill: with up to 64 row groups to a head they are counted in 32 bits.
constexpr int64_t kMostHeadTiles = (1 << 25) - 1;
constexpr float kLog2e = 1.4426950408889634f;

// f / 2 pi in units of 2^-64 of a turn, whole turns dropped, to the last of them (|f| <= kMostFreq): f = m 2^e with
// an integer m of 53 bits, times the first 128 bits of 1 / 2 pi.
constexpr double kMostFreq = 1024.0;
uint64_t turns(double f) {
  constexpr uint64_t kHi = 0x28be60db9391054aULL, kLo = 0x7f09d5f47d4d3770ULL;
  if (f == 0.0) return 0;
  int e;
  const uint64_t m = (uint64_t)ldexp(frexp(fabs(f), &e), 53);
  e -= 53;
  typedef unsigned __int128 u128;
  const u128 low = (u128)m * kLo;
  const u128 high = (u128)m * kHi + (uint64_t)(low >> 64);  // m / 2 pi, in units of 2^-64
  // high 2^e is f / 2 pi in units of 2^-64; e <= 11 - 53
  const uint64_t t = e <= -128 ? 0 : (uint64_t)(high >> -e);
  return f < 0 ? 0 - t : t;
}

// Rows of `width` elements, `stride` apart, `n` of them.
struct Rows {
  const char* p;
  int64_t stride, width, n;  // bytes
};
bool rows_ok(int64_t stride, int64_t width, int64_t n, int size) {
  // (no extent wraps around)
  return stride >= width && stride <= INT64_MAX / 8 / (n > 0 ? n : 1) && !(stride * size % 16);
}
// Whether two sets of rows share bytes. Of equal strides they may lie between one another.
bool share(const Rows& a, const Rows& b) {
  if (a.n <= 0 || b.n <= 0 || !a.width || !b.width) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t xe = x + (uintptr_t)((a.n - 1) * a.stride + a.width), ye = y + (uintptr_t)((b.n - 1) * b.stride + b.width);
  if (x >= ye || y >= xe) return false;
  if (a.stride != b.stride || (a.n == 1 && b.n == 1)) return true;
  const int64_t s = a.stride;
  int64_t d = (int64_t)((y > x ? y - x : x - y) % (uintptr_t)s);
  if (y < x && d) d = s - d;  // where b's rows begin behind a's, within a stride
  return d < a.width || d + b.width > s;
}

}  // namespace

extern "C" {

int kvarn_layout4(int head_dim, kvarn_layout4_t* out) {
  if (!out) return KVARN_ERR_NULL;
  if (!dim_ok(head_dim)) return KVARN_ERR_UNSUPPORTED;
  memset(out, 0, sizeof(*out));
  out->version = KVARN_LAYOUT4_VERSION;
  out->head_dim = head_dim;
  out->tile_tokens = KVARN_TILE_TOKENS;
  out->run_tokens = kvarn::kRun;
  out->group_channels = kvarn::kGroup4;
  out->run_bytes = 36LL * head_dim;
  out->record_bytes = kvarn::kRuns * out->run_bytes;
  out->off_k_codes = 0;
  out->off_v_codes = 16LL * head_dim;
  out->off_k_scale = 32LL * head_dim;
  out->off_v_scale = 34LL * head_dim;
  return KVARN_OK;
}

// What writing and reading check alike.
static int rows4_check(const kvarn::Rows4Args& a, const void* k, const void* v, const kvarn_layout4_t* layout) {
  if (!layout) return KVARN_ERR_NULL;
  if (!layout_ok(layout) || layout->head_dim != a.D) return KVARN_ERR_UNSUPPORTED;
  if (!io_ok(a.io) || !flags_ok(a.flags) || a.B < 0 || a.T < 0 || a.Hkv <= 0 || a.Hkv > 65535 || a.max_tiles < 0 ||
      a.max_tiles > kMostTiles || a.tiles_bytes < 0)
    return KVARN_ERR_BAD_ARG;
  if (a.B == 0 || a.T == 0) return KVARN_OK;
  const int64_t rows = (int64_t)a.B * a.T, width = (int64_t)a.Hkv * a.D;
  // a sequence's (row, head) pairs are counted in 32 bits
  if (a.B > 65535 || (int64_t)a.T * a.Hkv > 0x7fffff00) return KVARN_ERR_BAD_ARG;
  if (!k || !v || !a.first) return KVARN_ERR_NULL;
  if (a.max_tiles > 0 && (!a.tiles || !a.tile_table)) return KVARN_ERR_NULL;
  for (const int64_t s : {a.k_stride, a.v_stride}) {
    if (s * io_size(a.io) % 16) return KVARN_ERR_ALIGN;
    if (!rows_ok(s, width, rows, io_size(a.io))) return KVARN_ERR_BAD_ARG;
  }
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(a.tiles, 16) || !aligned(a.tile_table, 8) || !aligned(a.first, 4) ||
      !aligned(a.counts, 4))
    return KVARN_ERR_ALIGN;
  return KVARN_OK;
}

int kvarn_write_rows4(const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride, int io_type,
                      uint8_t* tiles, int64_t tiles_bytes, const int64_t* tile_table, const int32_t* lens,
                      const int32_t* counts, int B, int T, int Hkv, int head_dim, int max_tiles,
                      const kvarn_layout4_t* layout, unsigned launch_flags, kvarn_stream_t stream) {
  kvarn::Rows4Args a{k_new, v_new, nullptr, nullptr, tiles, tile_table, lens, counts, k_stride, v_stride,
                     tiles_bytes, io_type, B, T, Hkv, head_dim, max_tiles, launch_flags, nullptr};
  const int rc = rows4_check(a, k_new, v_new, layout);
  if (rc != KVARN_OK || B == 0 || T == 0) return rc;
  a.err = kvarn::device_error_word();
  return from_cuda(kvarn::launch_write4(a, (cudaStream_t)stream));
}

int kvarn_read_rows4(const uint8_t* tiles, int64_t tiles_bytes, const int64_t* tile_table, const int32_t* first,
                     const int32_t* counts, void* k_out, int64_t k_stride, void* v_out, int64_t v_stride, int io_type,
                     int B, int T, int Hkv, int head_dim, int max_tiles, const kvarn_layout4_t* layout,
                     unsigned launch_flags, kvarn_stream_t stream) {
  kvarn::Rows4Args a{nullptr, nullptr, k_out, v_out, const_cast<uint8_t*>(tiles), tile_table, first, counts,
                     k_stride, v_stride, tiles_bytes, io_type, B, T, Hkv, head_dim, max_tiles, launch_flags, nullptr};
  const int rc = rows4_check(a, k_out, v_out, layout);
  if (rc != KVARN_OK || B == 0 || T == 0) return rc;
  const int64_t rows = (int64_t)B * T, size = io_size(io_type), width = (int64_t)Hkv * head_dim * size;
  if (share(Rows{static_cast<const char*>(k_out), k_stride * size, width, rows},
            Rows{static_cast<const char*>(v_out), v_stride * size, width, rows}))
    return KVARN_ERR_BAD_ARG;
  a.err = kvarn::device_error_word();
  return from_cuda(kvarn::launch_read4(a, (cudaStream_t)stream));
}

static int decode4_check(int B, int Hq, int Hkv, int D, int max_tiles) {
  const int rc = heads_ok(Hq, Hkv, D);
  if (rc != KVARN_OK) return rc;
  if (B < 0 || max_tiles < 0 || B > 65535 || max_tiles > kMostTiles) return KVARN_ERR_BAD_ARG;
  // the merge grid's first dimension and the count of all tiles stay in range
  if ((int64_t)Hkv * ((max_tiles + 255) / 256) + Hq > 0x7fffffff) return KVARN_ERR_BAD_ARG;
  if (max_tiles > 0 && (int64_t)B * Hkv > 0x7fffffff / max_tiles) return KVARN_ERR_BAD_ARG;
  return KVARN_OK;
}

int kvarn_decode4_workspace_bytes(int B, int Hq, int Hkv, int head_dim, int max_tiles, size_t* bytes) {
  if (!bytes) return KVARN_ERR_NULL;
  const int rc = decode4_check(B, Hq, Hkv, head_dim, max_tiles);
  if (rc != KVARN_OK) return rc;
  kvarn::Decode4Plan p;
  kvarn::decode4_plan(B, Hq, Hkv, head_dim, max_tiles, &p);
  *bytes = p.ws_bytes;
  return KVARN_OK;
}

int kvarn_decode_attention4(const void* q, int io_type, const uint8_t* tiles, int64_t tiles_bytes,
                            const int64_t* tile_table, const int32_t* lens, int B, int Hq, int Hkv, int head_dim,
                            int max_tiles, float softmax_scale, const kvarn_layout4_t* layout, const float* mass_in,
                            float* mass_out, void* ws, size_t ws_bytes, void* out, unsigned launch_flags,
                            kvarn_stream_t stream) {
  const int rc = decode4_check(B, Hq, Hkv, head_dim, max_tiles);
  if (rc != KVARN_OK) return rc;
  if (!flags_ok(launch_flags) || tiles_bytes < 0 || !io_ok(io_type)) return KVARN_ERR_BAD_ARG;
  if (!layout) return KVARN_ERR_NULL;
  if (!layout_ok(layout) || layout->head_dim != head_dim) return KVARN_ERR_UNSUPPORTED;
  if (mass_in && !mass_out) return KVARN_ERR_BAD_ARG;
  if (!isfinite(softmax_scale)) return KVARN_ERR_BAD_ARG;
  if (B == 0) return KVARN_OK;
  if (!q || !out || !lens) return KVARN_ERR_NULL;
  if (max_tiles > 0 && (!tiles || !tile_table)) return KVARN_ERR_NULL;
  kvarn::Decode4Plan p;
  kvarn::decode4_plan(B, Hq, Hkv, head_dim, max_tiles, &p);
  const size_t need = mass_out ? p.ws_bytes : p.off_tile;  // (the tiles' weights are the workspace's last part)
  if (need > 0 && !ws) return KVARN_ERR_NULL;
  if (ws_bytes < need) return KVARN_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(tiles, 16) || !aligned(ws, 256) || !aligned(tile_table, 8) ||
      !aligned(lens, 4) || !aligned(mass_in, 4) || !aligned(mass_out, 4))
    return KVARN_ERR_ALIGN;
  const int64_t n_mass = 4LL * B * Hkv * max_tiles;
  if (mass_in && mass_in != mass_out &&
      share(Rows{reinterpret_cast<const char*>(mass_in), n_mass, n_mass, 1},
            Rows{reinterpret_cast<const char*>(mass_out), n_mass, n_mass, 1}))
    return KVARN_ERR_BAD_ARG;
  const kvarn::Decode4Args a{q, tiles, tile_table, lens, mass_in, mass_out, out, tiles_bytes, io_type, B, Hq, Hkv,
                             Hq / Hkv, head_dim, max_tiles, softmax_scale * kLog2e, launch_flags,
                             kvarn::device_error_word()};
  return from_cuda(kvarn::launch_decode4(p, a, ws, (cudaStream_t)stream));
}

int kvarn_prefill4_workspace_bytes(int C, int n_tiles, int Hq, int Hkv, int head_dim, size_t* bytes) {
  if (!bytes) return KVARN_ERR_NULL;
  const int rc = heads_ok(Hq, Hkv, head_dim);
  if (rc != KVARN_OK) return rc;
  if (C < 0 || n_tiles < 0 || n_tiles > kMostTiles || (int64_t)Hkv * n_tiles > kMostHeadTiles) return KVARN_ERR_BAD_ARG;
  *bytes = kvarn::prefill4_ws_bytes(C, n_tiles, Hq, Hkv, head_dim);
  return KVARN_OK;
}

int kvarn_prefill_attention4(const void* q_chunk, int io_type, int C, int64_t pos0, const uint8_t* tiles,
                             int64_t tiles_bytes, const int64_t* tile_table, int table_stride, int Hq, int Hkv,
                             int head_dim, float softmax_scale, const kvarn_layout4_t* layout, void* ws,
                             size_t ws_bytes, void* out, kvarn_stream_t stream) {
  const int rc = heads_ok(Hq, Hkv, head_dim);
  if (rc != KVARN_OK) return rc;
  if (!layout) return KVARN_ERR_NULL;
  if (!layout_ok(layout) || layout->head_dim != head_dim) return KVARN_ERR_UNSUPPORTED;
  if (!io_ok(io_type) || C < 0 || pos0 < 0 || table_stride < 0 || table_stride > kMostTiles || tiles_bytes < 0 ||
      !isfinite(softmax_scale))
    return KVARN_ERR_BAD_ARG;
  if (pos0 > (int64_t)KVARN_TILE_TOKENS * table_stride - C) return KVARN_ERR_BAD_ARG;
  if (C == 0) return KVARN_OK;
  if (!q_chunk || !out || !ws || !tiles || !tile_table) return KVARN_ERR_NULL;
  const int n_tiles = (int)((pos0 + C - 1) / KVARN_TILE_TOKENS + 1);
  if ((int64_t)Hkv * n_tiles > kMostHeadTiles) return KVARN_ERR_BAD_ARG;
  if (ws_bytes < kvarn::prefill4_ws_bytes(C, n_tiles, Hq, Hkv, head_dim)) return KVARN_ERR_WORKSPACE;
  if (!aligned(q_chunk, 16) || !aligned(out, 16) || !aligned(tiles, 16) || !aligned(ws, 256) || !aligned(tile_table, 8))
    return KVARN_ERR_ALIGN;
  const kvarn::Prefill4Args a{q_chunk, tiles, tile_table, static_cast<uint8_t*>(ws), out, tiles_bytes, (int)pos0, io_type,
                              C, Hq, Hkv, Hq / Hkv, head_dim, table_stride, softmax_scale * kLog2e,
                              kvarn::device_error_word()};
  return from_cuda(kvarn::launch_prefill4(a, (cudaStream_t)stream));
}

int kvarn_rotary(int rotary_dim, int pairing, const double* inv_freq, const uint8_t* pair_axis, int n_axes,
                 kvarn_rotary_t* out) {
  if (!out || !inv_freq) return KVARN_ERR_NULL;
  if (rotary_dim < 16 || rotary_dim > 256 || rotary_dim % 16) return KVARN_ERR_UNSUPPORTED;
  if ((pairing != KVARN_PAIRS_HALVES && pairing != KVARN_PAIRS_ADJACENT) || n_axes < 1 || n_axes > 4)
    return KVARN_ERR_BAD_ARG;
  const int pairs = rotary_dim / 2;
  for (int i = 0; i < pairs; ++i)
    if (!(fabs(inv_freq[i]) <= kMostFreq) || (pair_axis && pair_axis[i] >= n_axes)) return KVARN_ERR_BAD_ARG;
  memset(out, 0, sizeof(*out));
  out->version = KVARN_ROTARY_VERSION;
  out->rotary_dim = rotary_dim;
  out->pairing = pairing;
  out->n_axes = n_axes;
  for (int i = 0; i < pairs; ++i) {
    out->turn[i] = turns(inv_freq[i]);
    out->axis[i] = pair_axis ? pair_axis[i] : 0;
  }
  return KVARN_OK;
}

int kvarn_norm_rotate(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int io_type, int64_t n_tokens,
                      int Hq, int Hkv, int head_dim, const void* q_weight, const void* k_weight, float eps,
                      const int64_t* positions, const kvarn_rotary_t* rotary, int hadamard, void* q_out,
                      int64_t q_out_stride, void* k_out, int64_t k_out_stride, unsigned launch_flags,
                      kvarn_stream_t stream) {
  if (!dim_ok(head_dim)) return KVARN_ERR_UNSUPPORTED;
  if (!io_ok(io_type) || !flags_ok(launch_flags) || n_tokens < 0 || n_tokens > 0x7fffffff || Hq <= 0 || Hkv < 0 ||
      Hq > 65535 || Hkv > 65535 || eps != eps || eps > 3.4e38f)
    return KVARN_ERR_BAD_ARG;
  if (eps < 0 && (q_weight || k_weight)) return KVARN_ERR_BAD_ARG;
  if (Hkv == 0 && (k || k_out || k_weight)) return KVARN_ERR_BAD_ARG;
  if (rotary) {  // a plan that this library made
    if (rotary->version != KVARN_ROTARY_VERSION || rotary->rotary_dim < 16 || rotary->rotary_dim > head_dim ||
        rotary->rotary_dim % 16 || (rotary->pairing != KVARN_PAIRS_HALVES && rotary->pairing != KVARN_PAIRS_ADJACENT) ||
        rotary->n_axes < 1 || rotary->n_axes > 4)
      return KVARN_ERR_UNSUPPORTED;
    for (int i = 0; i < rotary->rotary_dim / 2; ++i)
      if (rotary->axis[i] >= rotary->n_axes) return KVARN_ERR_UNSUPPORTED;
  }
  if (n_tokens == 0) return KVARN_OK;
  if (!q || !q_out || (Hkv > 0 && (!k || !k_out)) || (rotary && !positions)) return KVARN_ERR_NULL;
  const int size = io_size(io_type);
  const int64_t wq = (int64_t)Hq * head_dim, wk = (int64_t)Hkv * head_dim;
  const int64_t strides[4] = {q_stride, q_out_stride, Hkv ? k_stride : 0, Hkv ? k_out_stride : 0};
  for (int i = 0; i < 4; ++i) {
    if (strides[i] * size % 16) return KVARN_ERR_ALIGN;
    if (!rows_ok(strides[i], i < 2 ? wq : wk, n_tokens, size)) return KVARN_ERR_BAD_ARG;
  }
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(positions, 8))
    return KVARN_ERR_ALIGN;
  auto rows = [&](const void* p, int64_t stride, int64_t width) {
    return Rows{static_cast<const char*>(p), stride * size, width * size, n_tokens};
  };
  const Rows in[2] = {rows(q, q_stride, wq), rows(k, k_stride, wk)};
  const Rows to[2] = {rows(q_out, q_out_stride, wq), rows(k_out, k_out_stride, wk)};
  const bool place[2] = {q_out == q && q_out_stride == q_stride, Hkv && k_out == k && k_out_stride == k_stride};
  if (share(to[0], to[1])) return KVARN_ERR_BAD_ARG;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (!(i == j && place[i]) && share(to[i], in[j])) return KVARN_ERR_BAD_ARG;
  const int axes = rotary ? rotary->n_axes : 0;
  const Rows others[3] = {Rows{reinterpret_cast<const char*>(positions), 0, 8 * n_tokens * axes, 1},
                          Rows{static_cast<const char*>(q_weight), 0, q_weight ? (int64_t)head_dim * size : 0, 1},
                          Rows{static_cast<const char*>(k_weight), 0, k_weight ? (int64_t)head_dim * size : 0, 1}};
  for (const Rows& t : to)
    for (const Rows& o : others)
      if (share(t, o)) return KVARN_ERR_BAD_ARG;
  const kvarn::RopeArgs a{q, k, q_out, k_out, q_weight, k_weight, positions, q_stride, k_stride, q_out_stride,
                          k_out_stride, n_tokens, io_type, Hq, Hkv, head_dim, hadamard != 0, eps, launch_flags};
  return from_cuda(kvarn::launch_norm_rotate(a, rotary, (cudaStream_t)stream));
}

}  // extern "C"
