// Shared pieces of the serving kernels (fa_cache.cu, fa_extend*.cu): the ragged
// batch, the paged cache, E4M3 rows with a power-of-two factor.
#pragma once

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_serving.h"

namespace fa {

constexpr int kPage = 128;   // keys per page

// A batch of B sequences with packed new tokens, and where its cache lives.
struct Ragged {
  int B, T;
  int H_kv, num_pages, max_pages;
  const int* cu;       // [B + 1]
  const int* lens;     // [B]
  const int* table;    // [B][max_pages]
};

// cu_seqlens and seqlens_k as the entry points define them: clamped, so that no value they
// may hold leads out of the tensors (decreasing ones: counts are cut at 0 below). (A length of max_pages * 128 + T puts
// all of a batch's tokens past the table, as any larger one does.)
__device__ __forceinline__ int cu_at(const Ragged& r, int b) { return min(max(__ldg(r.cu + b), 0), r.T); }
__device__ __forceinline__ int len_at(const Ragged& r, int b) {
  return min(max(__ldg(r.lens + b), 0), r.max_pages * kPage + r.T);
}
// Page of table entry `i` of sequence b, -1 when it lies outside the cache.
__device__ __forceinline__ int page_at(const Ragged& r, int b, int i) {
  const int pg = __ldg(r.table + (size_t)b * r.max_pages + i);
  return pg >= 0 && pg < r.num_pages ? pg : -1;
}

// 2^(byte - 127) in FP32 (byte 0: the subnormal 2^-127; 255: NaN, the row is).
__device__ __forceinline__ float exp_factor(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Two E4M3 codes (low byte first) widened to FP16, exactly (0x7F / 0xFF: NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two_codes));
  return r;
}
// Four codes to two pairs, lowest byte first.
__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// 1-D bulk copy global -> shared, counted on an mbarrier (16-byte aligned, a
// multiple of 16 bytes).
__device__ __forceinline__ void bulk_copy_1d(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4u(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ---- attention of new tokens over the cache (fa_extend_paged)
struct ExtendParams {
  Ragged r;
  int H_q, G, max_q;   // G = H_q / H_kv; tokens past max_q of a sequence are not computed
  // a batch that both kernels share: few > 0: only sequences of at most `few` new tokens;
  // few < 0: only those of more than -few; 0: all
  int few;
  int window, sinks;   // window 0: no window
  float c;             // scale * log2(e)
  const uint16_t* q;   // [T][H_q][d], tokens q_stride elements apart
  long long q_stride;
  void* o;             // [T][H_q][d]
  float* lse;          // [T][H_q] or nullptr
  const uint8_t *k_exp, *v_exp;   // E4M3 caches
  float* part_o;       // partials of split key ranges
  float* part_ml;
  int4* cuts;          // few rows: what the merge has to do after each CTA
  int* status;
};

// The tiles of 128 keys that query positions [p0, p1) (p1 > p0) see, of the first `tiles`: the
// sink tiles [0, n_sink), then [lo, hi). Positions below 0 or past those tiles see nothing.
struct KeyTiles {
  int n_sink, lo, hi;
  __device__ __forceinline__ int count() const { return n_sink + hi - lo; }
  __device__ __forceinline__ int tile(int k) const { return k < n_sink ? k : lo + (k - n_sink); }
};
__device__ __forceinline__ KeyTiles key_tiles_of(int p0, int p1, int window, int sinks, int tiles = 0x7FFFFFFF) {
  if (p0 / kPage >= tiles) return KeyTiles{0, 0, 0};
  KeyTiles kt;
  kt.hi = min((max(p1, 0) + kPage - 1) / kPage, tiles);
  kt.lo = window > 0 ? min(max(p0 - window + 1, 0) / kPage, kt.hi) : 0;
  kt.n_sink = window > 0 ? min((sinks + kPage - 1) / kPage, kt.lo) : 0;
  return kt;
}

// Sequence b's new tokens: rows t0 .. t0 + n - 1 of the packed batch are computed
// (n <= max_q); token t stands at position p0 + t; the sequence holds `len` keys, or as
// many as its table has room for.
struct SeqTokens {
  int t0, n, p0, len;
};
__device__ __forceinline__ SeqTokens seq_tokens(const ExtendParams& p, int b) {
  const Ragged& r = p.r;
  SeqTokens s;
  s.t0 = cu_at(r, b);
  const int all = max(cu_at(r, b + 1) - s.t0, 0);
  s.n = (p.few > 0 && all > p.few) || (p.few < 0 && all <= -p.few) ? 0 : min(all, p.max_q);
  s.len = len_at(r, b);
  s.p0 = s.len - all;
  return s;
}

// fa_extend_few.cu: at most kDecodeMaxRows rows per KV head (G * max_q), any lengths.
inline int few_groups(const ExtendParams& p) { return p.G * p.max_q <= 8 ? 1 : 2; }   // groups of 8 rows
int few_ctas(bool fp8, int groups);
cudaError_t launch_extend_few(int d, int dtype, int format, const CUtensorMap& tk, const CUtensorMap& tv,
                              const ExtendParams& p, cudaStream_t stream);

// fa_extend_tile.cu: any number of rows, 128-row tiles of packed (token, query head)
// rows; a ragged batch over pages, or uniform sequences over contiguous K and V.
constexpr int kTileMaxSeqs = 512;   // sequences one launch plans for
struct TileParams {
  ExtendParams e;      // e.r.table == nullptr: contiguous K and V, B sequences of N_q queries and N_k keys
  int N_q, N_k;
  int TQ;              // tokens per 128-row tile: 128 / G
  int sms;             // SMs of the device
  int grid;            // CTAs of the launch: at least the items of any plan
  int kv_bytes;        // K and V bytes per key of one KV head
  int key_tiles;       // tiles that the block table has room for (contiguous: no bound)
  int* cut;            // the plan's longest part, for the merge kernel
  int max_split_items; // 0: no key range is split
  long long o_b, o_t, o_h, o_g;   // element strides of o (lse: the same over d) by batch, token, KV head, query head
};
cudaError_t launch_tile(int d, int dtype, int format, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const TileParams& p, cudaStream_t stream);

// fa_extend.cu: how a tile launch runs (fills grid, kv_bytes, max_split_items): false when
// it is too large. Its workspace (0: none), and where that goes in the parameters.
bool tile_setup(TileParams& t, int d, int format);
size_t tile_workspace(const TileParams& t, int d);
void tile_use(TileParams& t, int d, void* ws);

// host-side checks shared by the serving entry points (fa_cache.cu)
bool ptr_aligned(const void* p, uintptr_t a);
bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb);
// Sizes of a ragged batch over a paged cache: fa_status code.
int check_ragged(int B, int T, int H_kv, int num_pages, int max_pages, int d, int dtype, int cache_format);

}  // namespace fa
