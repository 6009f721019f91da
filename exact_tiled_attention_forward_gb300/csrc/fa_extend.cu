// fa_extend_paged: checks, tensor maps, and which kernel runs.
#include "fa_serving.cuh"

#include <cmath>

namespace fa {

// Key ranges are cut only where that can pay for a second kernel (5 us or so): fewer units
// (2 TQ tokens of one KV head) than SMs and more than 8 key tiles (1.5 us each) in one, or
// up to 8 units an SM, of more than 32 tiles.
bool tile_setup(TileParams& t, int d, int format) {
  const Ragged& r = t.e.r;
  const bool paged = r.table != nullptr;
  const long long most_tokens = (long long)r.B * (paged ? t.e.max_q : t.N_q);   // of one launch
  const long long tokens = paged && r.T < most_tokens ? r.T : most_tokens;
  const long long U = 2 * t.TQ;
  const long long sure = (tokens + U - 1) / U * r.H_kv;            // units, at least (without padding rows)
  const long long units = (tokens / U + r.B) * r.H_kv;             // and at most
  if (units >= (1ll << 27)) return false;
  const long long keys = paged ? (long long)r.max_pages * kPage : t.N_k;
  long long tiles = (keys + kPage - 1) / kPage;
  if (t.e.window > 0) {
    const long long band = (t.e.window + U) / kPage + 2 + (t.e.sinks + kPage - 1) / kPage;
    tiles = tiles < band ? tiles : band;
  }
  const long long cap = 8ll * t.sms;
  t.max_split_items = 0;
  if ((sure < t.sms && tiles > 8) || (sure < cap && tiles > 32))
    t.max_split_items = (int)(16 * units < cap ? 16 * units : cap);
  t.grid = (int)(units > t.max_split_items ? units : t.max_split_items);
  t.kv_bytes = 2 * d * (format == FA_CACHE_E4M3 ? 1 : 2);
  t.key_tiles = paged ? r.max_pages : 0x7FFFFFFF;
  return true;
}

size_t tile_workspace(const TileParams& t, int d) {
  return t.max_split_items == 0 ? 0 : (size_t)t.max_split_items * kBlockRows * ((size_t)d + 2) * 4 + 16;
}

void tile_use(TileParams& t, int d, void* ws) {
  t.e.part_o = static_cast<float*>(ws);
  t.e.part_ml = t.e.part_o + (size_t)t.max_split_items * kBlockRows * d;
  t.cut = reinterpret_cast<int*>(t.e.part_ml + (size_t)t.max_split_items * kBlockRows * 2);
}

namespace {

int extend_impl(const void* q, const void* kc, const void* vc, const uint8_t* ke, const uint8_t* ve, const int* table,
                const int* cu, const int* lens, void* o, float* lse, int B, int T, int max_q, int H_q, int H_kv,
                int num_pages, int max_pages, int d, long long q_stride, int window, int sinks, float scale, int dtype,
                int format, cudaStream_t strm) {
  int st = check_ragged(B, T, H_kv, num_pages, max_pages, d, dtype, format);
  if (st != FA_OK) return st;
  if (max_q < 0 || H_q < 1 || H_q % H_kv != 0 || window < 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  const int G = H_q / H_kv;
  if (G > kPage) return FA_ERR_UNSUPPORTED;   // the query heads of a KV head fill one tile at most
  const long long width = (long long)H_q * d;
  if (q_stride < width || q_stride % 8 != 0 || q_stride > (1ll << 36)) return FA_ERR_INVALID_ARG;
  if ((long long)T * H_q >= (1ll << 31) || (long long)B * max_pages >= (1ll << 31) / H_kv)
    return FA_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || max_q == 0) return FA_OK;   // nothing to write
  const bool fp8 = format == FA_CACHE_E4M3;
  if (!q || !kc || !vc || !table || !cu || !lens || !o) return FA_ERR_INVALID_ARG;
  if (fp8 ? (!ke || !ve) : (ke || ve)) return FA_ERR_INVALID_ARG;
  const size_t cache_rows = (size_t)num_pages * H_kv * kPage;
  const size_t cb = cache_rows * d * (fp8 ? 1 : 2), eb = fp8 ? cache_rows : 0;
  const void* ptr[10] = {o, lse, q, kc, vc, ke, ve, table, cu, lens};
  const size_t len[10] = {(size_t)T * width * 2, lse ? (size_t)T * H_q * 4 : 0, ((size_t)(T - 1) * q_stride + width) * 2,
                          cb, cb, eb, eb, (size_t)B * max_pages * 4, ((size_t)B + 1) * 4, (size_t)B * 4};
  for (int i = 0; i < 10; ++i)
    if (!ptr_aligned(ptr[i], i < 7 && i != 1 ? 16 : 4)) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    for (int j = i + 1; j < 10; ++j)
      if (ranges_overlap(ptr[i], len[i], ptr[j], len[j])) return FA_ERR_INVALID_ARG;
  st = check_current_device(ptr, 10);
  if (st != FA_OK) return st;

  ExtendParams p{};
  p.r = Ragged{B, T, H_kv, num_pages, max_pages, cu, lens, table};
  p.H_q = H_q;
  p.G = G;
  p.max_q = max_q < T ? max_q : T;
  // a window that reaches past every position is none
  p.window = window < max_pages * kPage ? window : 0;
  p.sinks = sinks < max_pages * kPage ? sinks : max_pages * kPage;
  p.c = scale * 1.4426950408889634f;
  p.q = static_cast<const uint16_t*>(q);
  p.q_stride = q_stride;
  p.o = o;
  p.lse = lse;
  p.k_exp = ke;
  p.v_exp = ve;
  p.status = device_status_ptr();
  if (!p.status) return cuda_fail(cudaGetLastError());
  CUtensorMap tk, tv;
  const uint64_t slabs = (uint64_t)num_pages * H_kv;   // one per (page, KV head)
  if (fp8 ? (!make_tmap_u8_3d(&tk, kc, d, kPage, slabs, kPage) || !make_tmap_u8_3d(&tv, vc, d, kPage, slabs, kPage))
          : (!make_tmap_bf16_3d(&tk, kc, d, kPage, slabs, d, kPage) ||
             !make_tmap_bf16_3d(&tv, vc, d, kPage, slabs, d, kPage)))
    return cuda_fail(cudaErrorInvalidValue);
  // Which kernel: the few-row kernel when max_q allows it, else tiles. In tiles a single
  // token costs what 128 rows do, and over E4M3 pages that is the widening of every tile
  // of its keys. So over E4M3 pages, when the counts say that most sequences bring a token or
  // two beside a few chunks (continuous batching), each kernel takes its own: a chunk of
  // 1000 beside 15 single tokens runs in 94 us instead of 118, one of 512 beside 63 in 80
  // instead of 141. The other kernel's launch costs 6 to 12 us, about 10 ns for each of
  // 1000 key tiles: hence the bound on those. Over 16-bit pages the two came out even
  // (111 against 106 us, 154 against 170), so tiles take all.
  const bool tiles = (long long)G * p.max_q > kDecodeMaxRows;
  const int small = G <= 8 ? 8 / G : kDecodeMaxRows / G;   // new tokens the few-row kernel takes then
  const long long chunks = ((long long)T + p.max_q - 1) / p.max_q;   // at least
  const long long seen = p.window > 0 ? ((long long)p.window + p.sinks) / kPage + 2 : max_pages;
  const bool both = tiles && fp8 && small > 0 && B >= 2 * chunks + 2 &&
                    (B - chunks) * H_kv * (seen < max_pages ? seen : max_pages) >= 16ll * num_sms();
  ExtendParams pf = p;
  size_t few_bytes = 0, slots = 0;
  int ctas = 0;
  if (!tiles || both) {
    if (both) {
      pf.few = small;
      pf.max_q = small;
    }
    // two partials of 16 rows for each CTA (O, and m and l), and its entry for the merge
    ctas = few_ctas(fp8, few_groups(pf));
    slots = (size_t)ctas * 2 * 16;
    few_bytes = (slots * (d + 2) * 4 + (size_t)ctas * sizeof(int4) + 255) / 256 * 256;
  }
  TileParams t{};
  CUtensorMap tq;
  size_t tile_bytes = 0;
  if (tiles) {
    // 128-row tiles of TQ tokens x G heads
    t.e = p;
    if (both) t.e.few = -small;
    t.e.r.B = B < kTileMaxSeqs ? B : kTileMaxSeqs;
    t.TQ = kPage / G;
    t.sms = num_sms();
    t.o_t = width;
    t.o_h = (long long)G * d;
    t.o_g = d;
    if (!tile_setup(t, d, format)) return FA_ERR_INVALID_ARG;
    tile_bytes = tile_workspace(t, d);
    const uint64_t dims[5] = {(uint64_t)d, (uint64_t)G, (uint64_t)T, (uint64_t)H_kv, 1};
    const uint64_t str[4] = {(uint64_t)d * 2, (uint64_t)q_stride * 2, (uint64_t)G * d * 2, (uint64_t)q_stride * 2};
    if (!make_tmap_rows_5d(&tq, q, dims, str, (uint32_t)G, (uint32_t)t.TQ)) return cuda_fail(cudaErrorInvalidValue);
  }
  const WorkspaceSource& pool = pool_workspace();
  void* ws = nullptr;
  if (few_bytes + tile_bytes > 0) {
    st = pool.acquire(few_bytes + tile_bytes, strm, &ws);
    if (st != FA_OK) return st;
  }
  cudaError_t e = cudaSuccess;
  // a tile launch plans for kTileMaxSeqs sequences; more take several, in turn on one workspace
  for (int b0 = 0; tiles && b0 < B && e == cudaSuccess; b0 += kTileMaxSeqs) {
    t.e.r.B = B - b0 < kTileMaxSeqs ? B - b0 : kTileMaxSeqs;
    t.e.r.cu = cu + b0;
    t.e.r.lens = lens + b0;
    t.e.r.table = table + (size_t)b0 * max_pages;
    tile_use(t, d, static_cast<char*>(ws) + few_bytes);
    e = launch_tile(d, dtype, format, tq, tk, tv, t, strm);
  }
  if (few_bytes > 0 && e == cudaSuccess) {
    pf.cuts = static_cast<int4*>(ws);
    pf.part_o = reinterpret_cast<float*>(pf.cuts + ctas);
    pf.part_ml = pf.part_o + slots * d;
    e = launch_extend_few(d, dtype, format, tk, tv, pf, strm);
  }
  if (ws) pool.release(ws, strm);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace fa

extern "C" int fa_extend_paged(const void* q, const void* k_cache, const void* v_cache, const unsigned char* k_exp,
                               const unsigned char* v_exp, const int* block_table, const int* cu_seqlens,
                               const int* seqlens_k, void* o, float* lse, int B, int T, int max_q, int H_q, int H_kv,
                               int num_pages, int max_pages, int d, long long q_stride, int window, int sinks,
                               float scale, int dtype, int cache_format, void* stream) {
  return fa::extend_impl(q, k_cache, v_cache, k_exp, v_exp, block_table, cu_seqlens, seqlens_k, o, lse, B, T, max_q,
                         H_q, H_kv, num_pages, max_pages, d, q_stride, window, sinks, scale, dtype, cache_format,
                         static_cast<cudaStream_t>(stream));
}
