// kvarn8_abi.cu -- the extern "C" entry points of the 8-bit cache and of eviction: arguments
// are checked on the host, and nothing is enqueued when they are wrong.
#include <stdint.h>
#include <string.h>

#include "cache8.cuh"

namespace {

bool dim_ok(int D) { return D == 64 || D == 128 || D == 256; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA; }
bool io_ok(int io) { return io == KVARN_IO_F32 || io == KVARN_IO_F16 || io == KVARN_IO_BF16; }
bool flags_ok(unsigned f) {
  return !(f & ~(KVARN_LAUNCH_PDL | KVARN_LAUNCH_PREFETCH)) &&
         !((f & KVARN_LAUNCH_PREFETCH) && !(f & KVARN_LAUNCH_PDL));
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// A layout handed back by the caller must be one this library produced.
bool layout_ok(const kvarn_layout8_t* L) {
  kvarn_layout8_t ref;
  return kvarn_layout8(L->head_dim, L->code_format, L->block_tokens, &ref) == KVARN_OK &&
         memcmp(&ref, L, sizeof(ref)) == 0;
}

int heads_ok(int Hq, int Hkv, int D) {
  if (!dim_ok(D)) return KVARN_ERR_UNSUPPORTED;
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || Hkv > 65535) return KVARN_ERR_BAD_ARG;
  if (Hq / Hkv > 8) return KVARN_ERR_UNSUPPORTED;
  return KVARN_OK;
}

// Tiles of a head and window rows stay below this, so that the kernels' 32-bit counts of them hold.
constexpr int kMost = 1 << 29;

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace

extern "C" {

int kvarn_layout8(int head_dim, int code_format, int block_tokens, kvarn_layout8_t* out) {
  if (!out) return KVARN_ERR_NULL;
  if (!dim_ok(head_dim) || (code_format != KVARN_CODE8_I8 && code_format != KVARN_CODE8_E4M3) ||
      (block_tokens != 16 && block_tokens != 32 && block_tokens != 64 && block_tokens != 128))
    return KVARN_ERR_UNSUPPORTED;
  memset(out, 0, sizeof(*out));
  out->version = KVARN_LAYOUT8_VERSION;
  out->head_dim = head_dim;
  out->tile_tokens = KVARN_TILE_TOKENS;
  out->code_format = code_format;
  out->block_tokens = block_tokens;
  out->off_k_codes = 0;
  out->off_v_codes = (int64_t)KVARN_TILE_TOKENS * head_dim;
  out->off_k_scale = 2 * out->off_v_codes;
  out->off_v_scale = out->off_k_scale + 4 * kvarn::kGrps;
  out->record_bytes = out->off_k_scale + 128;
  return KVARN_OK;
}

// What compression and expansion check alike.
static int rows_check(const void* k, const void* v, int64_t row_stride, int64_t n_rows, const void* rows,
                      const void* tiles, int64_t tiles_bytes, const void* records, int64_t n_units,
                      const kvarn_layout8_t* layout) {
  if (!layout) return KVARN_ERR_NULL;
  if (!layout_ok(layout)) return KVARN_ERR_UNSUPPORTED;
  if (n_units < 0 || n_units > 0x3fffffff || n_rows < 0 || tiles_bytes < 0) return KVARN_ERR_BAD_ARG;
  if (n_units == 0) return KVARN_OK;
  if (!k || !v || !rows || !tiles || !records) return KVARN_ERR_NULL;
  if (row_stride < layout->head_dim || n_rows < KVARN_TILE_TOKENS || tiles_bytes < layout->record_bytes)
    return KVARN_ERR_BAD_ARG;
  if ((row_stride & 3) || !aligned(k, 16) || !aligned(v, 16) || !aligned(tiles, 16) || !aligned(rows, 8) ||
      !aligned(records, 8))
    return KVARN_ERR_ALIGN;
  return KVARN_OK;
}

int kvarn_compress_tile8(const float* k_raw, const float* v_raw, int64_t row_stride, int64_t n_rows,
                         const int64_t* src_row0, uint8_t* tiles, int64_t tiles_bytes,
                         const int64_t* dst_record, int64_t n_units, const kvarn_layout8_t* layout,
                         kvarn_stream_t stream) {
  const int rc = rows_check(k_raw, v_raw, row_stride, n_rows, src_row0, tiles, tiles_bytes, dst_record,
                            n_units, layout);
  if (rc != KVARN_OK || n_units == 0) return rc;
  return from_cuda(kvarn::launch_compress8(layout->head_dim, layout->code_format, layout->block_tokens, k_raw,
                                           v_raw, row_stride, n_rows, src_row0, tiles, tiles_bytes,
                                           dst_record, n_units, kvarn::device_error_word(),
                                           (cudaStream_t)stream));
}

int kvarn_expand_tile8(const uint8_t* tiles, int64_t tiles_bytes, const int64_t* src_record, float* k_out,
                       float* v_out, int64_t row_stride, int64_t n_rows, const int64_t* dst_row0,
                       int64_t n_units, const kvarn_layout8_t* layout, kvarn_stream_t stream) {
  const int rc = rows_check(k_out, v_out, row_stride, n_rows, dst_row0, tiles, tiles_bytes, src_record,
                            n_units, layout);
  if (rc != KVARN_OK || n_units == 0) return rc;
  return from_cuda(kvarn::launch_expand8(layout->head_dim, layout->code_format, tiles, tiles_bytes, src_record,
                                         k_out, v_out, row_stride, n_rows, dst_row0, n_units,
                                         kvarn::device_error_word(), (cudaStream_t)stream));
}

static int decode8_check(int B, int Hq, int Hkv, int D, int max_tiles, int win_capacity) {
  const int rc = heads_ok(Hq, Hkv, D);
  if (rc != KVARN_OK) return rc;
  if (B < 0 || max_tiles < 0 || win_capacity < 0 || B > 65535 || max_tiles > kMost || win_capacity > kMost)
    return KVARN_ERR_BAD_ARG;
  // the grids' first dimension and the workspace stay in range
  if ((int64_t)Hkv * ((max_tiles + 255) / 256) + Hq > 0x7fffffff) return KVARN_ERR_BAD_ARG;
  return KVARN_OK;
}

int kvarn_decode8_workspace_bytes(int B, int Hq, int Hkv, int head_dim, int max_tiles, int win_capacity,
                                  size_t* bytes) {
  if (!bytes) return KVARN_ERR_NULL;
  const int rc = decode8_check(B, Hq, Hkv, head_dim, max_tiles, win_capacity);
  if (rc != KVARN_OK) return rc;
  kvarn::Decode8Plan p;
  kvarn::decode8_plan(B, Hq, Hkv, head_dim, max_tiles, win_capacity, &p);
  *bytes = p.ws_bytes;
  return KVARN_OK;
}

int kvarn_decode_attention8(const void* q, int io_type, const uint8_t* tiles, int64_t tiles_bytes,
                            const int64_t* tile_table, const int32_t* n_tiles, const float* win_k,
                            const float* win_v, const int32_t* win_start, const int32_t* win_len,
                            int win_capacity, int B, int Hq, int Hkv, int head_dim, int max_tiles,
                            float softmax_scale, const kvarn_layout8_t* layout, const float* mass_in,
                            float* mass_out, void* ws, size_t ws_bytes, void* out, unsigned launch_flags,
                            kvarn_stream_t stream) {
  const int rc = decode8_check(B, Hq, Hkv, head_dim, max_tiles, win_capacity);
  if (rc != KVARN_OK) return rc;
  if (!flags_ok(launch_flags) || tiles_bytes < 0 || !io_ok(io_type)) return KVARN_ERR_BAD_ARG;
  if (!layout) return KVARN_ERR_NULL;
  if (!layout_ok(layout) || layout->head_dim != head_dim) return KVARN_ERR_UNSUPPORTED;
  if (mass_in && !mass_out) return KVARN_ERR_BAD_ARG;
  if (!(softmax_scale == softmax_scale)) return KVARN_ERR_BAD_ARG;
  if (B == 0) return KVARN_OK;
  if (!q || !out || !n_tiles) return KVARN_ERR_NULL;
  if (max_tiles > 0 && (!tiles || !tile_table)) return KVARN_ERR_NULL;
  if (win_capacity > 0 && (!win_k || !win_v || !win_start || !win_len)) return KVARN_ERR_NULL;
  kvarn::Decode8Plan p;
  kvarn::decode8_plan(B, Hq, Hkv, head_dim, max_tiles, win_capacity, &p);
  if (p.ws_bytes > 0 && !ws) return KVARN_ERR_NULL;
  if (ws_bytes < p.ws_bytes) return KVARN_ERR_WORKSPACE;
  if (!aligned(q, 16) || !aligned(out, 16) || (max_tiles > 0 && !aligned(tiles, 16)) ||
      (win_capacity > 0 && (!aligned(win_k, 16) || !aligned(win_v, 16))) || !aligned(ws, 256) ||
      !aligned(tile_table, 8) || !aligned(n_tiles, 4) || !aligned(win_start, 4) || !aligned(win_len, 4) ||
      !aligned(mass_in, 4) || !aligned(mass_out, 4))
    return KVARN_ERR_ALIGN;
  const size_t n_mass = (size_t)B * Hkv * max_tiles * sizeof(float);
  if (mass_in && mass_in != mass_out && overlap(mass_in, n_mass, mass_out, n_mass)) return KVARN_ERR_BAD_ARG;
  const kvarn::Decode8Args a{q, tiles, tile_table, n_tiles, win_k, win_v, win_start, win_len, mass_in, mass_out,
                             out, tiles_bytes, io_type, win_capacity, B, Hq, Hkv, Hq / Hkv, head_dim,
                             max_tiles, layout->code_format, softmax_scale * kLog2e, launch_flags,
                             kvarn::device_error_word()};
  return from_cuda(kvarn::launch_decode8(p, a, ws, (cudaStream_t)stream));
}

int kvarn_prefill8_workspace_bytes(int C, int n_tiles, int win_len, int Hq, int Hkv, int head_dim,
                                   size_t* bytes) {
  if (!bytes) return KVARN_ERR_NULL;
  const int rc = heads_ok(Hq, Hkv, head_dim);
  if (rc != KVARN_OK) return rc;
  if (C < 0 || n_tiles < 0 || win_len < 0 || n_tiles > kMost || win_len > kMost) return KVARN_ERR_BAD_ARG;
  *bytes = kvarn::prefill8_ws_bound(C, n_tiles, win_len, Hq, Hkv, head_dim);
  return KVARN_OK;
}

int kvarn_prefill_attention8(const void* q_chunk, int io_type, int C, int64_t pos0, const uint8_t* tiles,
                             int64_t tiles_bytes, const int64_t* tile_table, int table_stride, int n_tiles,
                             const float* win_k, const float* win_v, int win_start, int win_len,
                             int win_capacity, int Hq, int Hkv, int head_dim, float softmax_scale,
                             const kvarn_layout8_t* layout, void* ws, size_t ws_bytes, void* out,
                             kvarn_stream_t stream) {
  const int rc = heads_ok(Hq, Hkv, head_dim);
  if (rc != KVARN_OK) return rc;
  if (!layout) return KVARN_ERR_NULL;
  if (!layout_ok(layout) || layout->head_dim != head_dim) return KVARN_ERR_UNSUPPORTED;
  if (!io_ok(io_type) || C < 0 || pos0 < 0 || n_tiles < 0 || win_len < 0 || win_capacity < 0 ||
      tiles_bytes < 0 || table_stride < n_tiles || win_len > win_capacity || n_tiles > kMost ||
      win_capacity > kMost)
    return KVARN_ERR_BAD_ARG;
  if (pos0 > (int64_t)KVARN_TILE_TOKENS * n_tiles + win_len - C) return KVARN_ERR_BAD_ARG;
  if (!(softmax_scale == softmax_scale)) return KVARN_ERR_BAD_ARG;
  if (C == 0) return KVARN_OK;
  if (!q_chunk || !out || !ws) return KVARN_ERR_NULL;
  if (n_tiles > 0 && (!tiles || !tile_table)) return KVARN_ERR_NULL;
  if (win_len > 0 && (!win_k || !win_v)) return KVARN_ERR_NULL;
  if (ws_bytes < kvarn::prefill8_ws_bytes(C, n_tiles, win_len, Hq, Hkv, head_dim)) return KVARN_ERR_WORKSPACE;
  if (!aligned(q_chunk, 16) || !aligned(out, 16) || (n_tiles > 0 && !aligned(tiles, 16)) ||
      (win_len > 0 && (!aligned(win_k, 16) || !aligned(win_v, 16))) || !aligned(ws, 256) || !aligned(tile_table, 8))
    return KVARN_ERR_ALIGN;
  const int start = win_capacity > 0 ? (int)((((int64_t)win_start % win_capacity) + win_capacity) % win_capacity) : 0;
  const kvarn::Prefill8Args a{q_chunk, tiles, tile_table, win_k, win_v, static_cast<uint8_t*>(ws), out, pos0,
                              tiles_bytes, io_type, C, Hq, Hkv, Hq / Hkv, head_dim, layout->code_format,
                              n_tiles, table_stride, start, win_len, win_capacity, softmax_scale * kLog2e,
                              kvarn::device_error_word()};
  return from_cuda(kvarn::launch_prefill8(a, (cudaStream_t)stream));
}

int kvarn_evict_tiles(const int64_t* tile_table, const float* tile_mass, const int32_t* n_tiles,
                      int64_t* table_out, float* mass_out, int32_t* n_tiles_out, int64_t* evicted, int B,
                      int Hkv, int max_tiles, int keep, int sinks, int recent, unsigned launch_flags,
                      kvarn_stream_t stream) {
  if (B < 0 || B > 65535 || Hkv <= 0 || Hkv > 65535 || max_tiles < 0 || max_tiles > kMost || keep < 1 ||
      sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep || (launch_flags & ~KVARN_LAUNCH_PDL))
    return KVARN_ERR_BAD_ARG;
  if (B == 0) return KVARN_OK;
  if (!n_tiles || !n_tiles_out) return KVARN_ERR_NULL;
  if (max_tiles > 0 && (!tile_table || !tile_mass || !table_out || !mass_out)) return KVARN_ERR_NULL;
  if (!aligned(tile_table, 8) || !aligned(table_out, 8) || !aligned(evicted, 8) || !aligned(tile_mass, 4) ||
      !aligned(mass_out, 4) || !aligned(n_tiles, 4) || !aligned(n_tiles_out, 4))
    return KVARN_ERR_ALIGN;
  const size_t n = (size_t)B * Hkv * max_tiles, n8 = n * 8, n4 = n * 4, nb = 4 * (size_t)B;
  if ((table_out != tile_table && overlap(table_out, n8, tile_table, n8)) ||
      (mass_out != tile_mass && overlap(mass_out, n4, tile_mass, n4)) ||
      overlap(table_out, n8, tile_mass, n4) || overlap(table_out, n8, mass_out, n4) ||
      overlap(tile_table, n8, mass_out, n4) ||
      (n_tiles_out != n_tiles && overlap(n_tiles_out, nb, n_tiles, nb)))
    return KVARN_ERR_BAD_ARG;
  // the counts apart from what is written, and the written counts from what is read
  for (const int32_t* c : {n_tiles, (const int32_t*)n_tiles_out})
    if (overlap(c, nb, table_out, n8) || overlap(c, nb, mass_out, n4) || (evicted && overlap(c, nb, evicted, n8)))
      return KVARN_ERR_BAD_ARG;
  if (overlap(n_tiles_out, nb, tile_table, n8) || overlap(n_tiles_out, nb, tile_mass, n4)) return KVARN_ERR_BAD_ARG;
  if (evicted && (overlap(evicted, n8, tile_table, n8) || overlap(evicted, n8, table_out, n8) ||
                  overlap(evicted, n8, tile_mass, n4) || overlap(evicted, n8, mass_out, n4)))
    return KVARN_ERR_BAD_ARG;
  return from_cuda(kvarn::launch_evict(tile_table, tile_mass, n_tiles, table_out, mass_out, n_tiles_out,
                                       evicted, B, Hkv, max_tiles, keep, sinks, recent, launch_flags,
                                       (cudaStream_t)stream));
}

}  // extern "C"
