// fa_cache_append and fa_cache_read: new tokens' K and V into a paged cache, as
// they are or quantised to E4M3 with one power of two per row, and back.
//
// A row is one token of one KV head (d elements). Quantising it: with
// max|x| = m * 2^x, 1 <= m < 2, and 448 = 1.75 * 2^8 the largest E4M3 value, the
// smallest e with max|x| <= 448 * 2^e is x - 8 when m <= 1.75 and x - 7
// otherwise, read off the bits of the maximum. A power of two costs no precision
// against max|x| / 448 (E4M3 is a floating format: only its underflow moves, by
// less than one binade), takes one byte instead of four, makes x * 2^-e exact
// and leaves every stored value exactly representable in the 16-bit type, so
// attention over the codes is attention over a 16-bit cache of these values.
//
// Bound: HBM. Each row is read and written once: 2 d + d + 1 bytes either way.
// d / 8 lanes share a row, 16 bytes of the 16-bit side each, K and V of two rows in
// flight together; the row maximum is 3 or 4 shuffles. Measured (8 KV heads, d = 128, BF16 and
// E4M3): 45624 tokens appended in 55 us (281 MB, 5.1 TB/s; 65 us with the heads of a token side
// by side, whose codes lie 16 KB apart), 105261 read back in 105 us
// (648 MB, 6.2 TB/s; a copy makes 6.8). 16 tokens take 2.8 us, a launch. 16-bit caches of the same
// sizes: 57.9 us (374 MB, 6.5 TB/s), 128.6 us (862 MB, 6.7 TB/s), 2.5 us.
#include "fa_serving.cuh"

namespace fa {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kCuShared = 1025;   // cu_seqlens of up to 1024 sequences are staged in shared memory

struct CacheParams {
  Ragged r;
  const uint16_t *k_in, *v_in;       // append: new rows, tokens `k_stride` / `v_stride` elements apart
  long long k_stride, v_stride;
  uint16_t *k_out, *v_out;           // read: [T][H_kv][d]
  uint8_t *k_cache, *v_cache, *k_exp, *v_exp;
};

// The last b with cu[b] <= t (cu non-decreasing, cu[0] <= t): the sequence of token t.
template <typename F>
__device__ __forceinline__ int seq_of(int t, int B, F cu) {
  int lo = 0, hi = B;   // cu(lo) <= t < cu(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu(mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <Elem E>
__device__ __forceinline__ void widen8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E == Elem::F16) {
      const float2 f = f16x2_to_f32x2(u[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
}

// Eight elements of a row (the d / 8 lanes of the row hold the others): their
// codes, and the row's exponent byte.
template <int D, Elem E>
__device__ __forceinline__ uint2 quantise8(const uint4& w, uint32_t& byte) {
  float x[8];
  widen8<E>(w, x);
  // the maximum of the magnitudes as bit patterns: a NaN or an infinity (0x7F800000
  // and above) wins over every number
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int off = D / 16; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top >= 0x7F800000u) {
    byte = 255;
    return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
  // biased exponent of max|x|, less 8, plus 1 when its mantissa exceeds 1.75; at
  // least 7 (2^-120: below it the codes' own steps would leave the 16-bit range)
  const int eb = max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 7);
  byte = (uint32_t)eb;
  const float inv = __uint_as_float((uint32_t)(254 - eb) << 23);   // 2^(127 - eb)
  return make_uint2(pack4_e4m3(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    pack4_e4m3(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

template <Elem E>
__device__ __forceinline__ uint4 dequantise8(const uint2& codes, uint32_t byte) {
  const float f = exp_factor(byte);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = ((i < 2 ? codes.x : codes.y) >> (16 * (i & 1))) & 0xFFFFu;
    const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2(two));
    r[i] = pack2<E>(v.x * f, v.y * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A block takes one KV head of kRows * kUnroll consecutive tokens at a time, D / 8 lanes a
// row, looping over the grid: in the cache its rows lie together (whole pages' worth of
// codes, neighbouring exponent bytes), on the 16-bit side each is 256 or 128 bytes.
template <int D, Elem E, bool FP8, bool READ, int kUnroll>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_kernel(const CacheParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = kCacheThreads / kLanes;
  __shared__ int s_cu[kCuShared];
  const Ragged& r = p.r;
  const bool staged = r.B < kCuShared;
  if (staged) {
    for (int i = threadIdx.x; i <= r.B; i += kCacheThreads) s_cu[i] = cu_at(r, i);
    __syncthreads();
  }
  auto cu = [&](int i) { return staged ? s_cu[i] : cu_at(r, i); };
  const int first = cu(0), end = cu(r.B);
  const int c = threadIdx.x % kLanes;   // this lane's 8 elements of the row
  // (every lane of a warp runs the same trips: the row maximum is a warp shuffle)
  const int chunks = (r.T + kRows * kUnroll - 1) / (kRows * kUnroll);
  for (unsigned w = blockIdx.x; w < (unsigned)chunks * (unsigned)r.H_kv; w += gridDim.x) {
    const int chunk = (int)(w / (unsigned)r.H_kv), h = (int)(w - (unsigned)chunk * (unsigned)r.H_kv);
    int tok[kUnroll];
    bool live[kUnroll];
    long long at[kUnroll];   // cache row, -1: nowhere
    uint4 wk[kUnroll], wv[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      tok[x] = chunk * (kRows * kUnroll) + x * kRows + (int)threadIdx.x / kLanes;
      live[x] = tok[x] >= first && tok[x] < end;   // not padding
      wk[x] = wv[x] = make_uint4(0, 0, 0, 0);
      if (!READ && live[x]) {   // the loads go out before the look-ups that place them
        wk[x] = __ldcs(reinterpret_cast<const uint4*>(p.k_in + tok[x] * p.k_stride + (long long)h * D) + c);
        wv[x] = __ldcs(reinterpret_cast<const uint4*>(p.v_in + tok[x] * p.v_stride + (long long)h * D) + c);
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      at[x] = -1;
      if (live[x]) {
        const int b = seq_of(tok[x], r.B, cu);
        const int e = max(cu(b + 1), cu(b));
        const int pos = len_at(r, b) - (e - tok[x]);
        const int pg = pos >= 0 && pos < r.max_pages * kPage ? page_at(r, b, pos / kPage) : -1;
        if (pg >= 0) at[x] = ((long long)pg * r.H_kv + h) * kPage + pos % kPage;
      }
    }
    if constexpr (READ) {
      uint2 ck[kUnroll], cv[kUnroll];
      uint32_t ek[kUnroll], ev[kUnroll];
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        ck[x] = cv[x] = make_uint2(0, 0);
        ek[x] = ev[x] = 127;
        if (at[x] < 0) continue;
        if constexpr (FP8) {
          ck[x] = __ldcs(reinterpret_cast<const uint2*>(p.k_cache + at[x] * D) + c);
          cv[x] = __ldcs(reinterpret_cast<const uint2*>(p.v_cache + at[x] * D) + c);
          ek[x] = __ldg(p.k_exp + at[x]);
          ev[x] = __ldg(p.v_exp + at[x]);
        } else {
          wk[x] = __ldcs(reinterpret_cast<const uint4*>(p.k_cache + at[x] * (D * 2)) + c);
          wv[x] = __ldcs(reinterpret_cast<const uint4*>(p.v_cache + at[x] * (D * 2)) + c);
        }
      }
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        if (!live[x]) continue;
        if constexpr (FP8) {
          wk[x] = dequantise8<E>(ck[x], ek[x]);
          wv[x] = dequantise8<E>(cv[x], ev[x]);
        }
        const size_t row = ((size_t)tok[x] * r.H_kv + h) * D;
        __stcs(reinterpret_cast<uint4*>(p.k_out + row) + c, wk[x]);
        __stcs(reinterpret_cast<uint4*>(p.v_out + row) + c, wv[x]);
      }
    } else {
#pragma unroll
      for (int x = 0; x < kUnroll; ++x) {
        if constexpr (FP8) {
          uint32_t ek, ev;
          const uint2 ck = quantise8<D, E>(wk[x], ek);
          const uint2 cv = quantise8<D, E>(wv[x], ev);
          if (at[x] >= 0) {
            __stcs(reinterpret_cast<uint2*>(p.k_cache + at[x] * D) + c, ck);
            __stcs(reinterpret_cast<uint2*>(p.v_cache + at[x] * D) + c, cv);
            if (c == 0) {
              p.k_exp[at[x]] = (uint8_t)ek;
              p.v_exp[at[x]] = (uint8_t)ev;
            }
          }
        } else if (at[x] >= 0) {
          reinterpret_cast<uint4*>(p.k_cache + at[x] * (D * 2))[c] = wk[x];
          reinterpret_cast<uint4*>(p.v_cache + at[x] * (D * 2))[c] = wv[x];
        }
      }
    }
  }
}

template <bool READ>
cudaError_t launch_cache(const CacheParams& p, int d, int dtype, int format, cudaStream_t stream) {
  // small batches: a row at a time, over as many blocks as that makes; larger ones: two
  const int sms = num_sms();
  const int one = kCacheThreads / (d / 8);
  const bool small = (long long)p.r.T * p.r.H_kv <= 4ll * one * sms;
  const int rows = small ? one : 2 * one;
  const long long want = (long long)((p.r.T + rows - 1) / rows) * p.r.H_kv, most = 32ll * sms;
  const dim3 grid((unsigned)(want < most ? want : most)), block(kCacheThreads);
#define FA_CACHE_GO(DD, EE, FF)                                                                            \
  return small ? launch_kernel(fa_cache_kernel<DD, EE, FF, READ, 1>, grid, block, 0, stream, p)            \
               : launch_kernel(fa_cache_kernel<DD, EE, FF, READ, 2>, grid, block, 0, stream, p)
  const bool f16 = dtype == FA_DTYPE_FP16;
  if (format == FA_CACHE_E4M3) {
    if (d == 128) {
      if (f16) FA_CACHE_GO(128, Elem::F16, true);
      FA_CACHE_GO(128, Elem::BF16, true);
    }
    if (f16) FA_CACHE_GO(64, Elem::F16, true);
    FA_CACHE_GO(64, Elem::BF16, true);
  }
  // 16-bit caches are copied: the element type does not matter
  if (d == 128) FA_CACHE_GO(128, Elem::BF16, false);
  FA_CACHE_GO(64, Elem::BF16, false);
#undef FA_CACHE_GO
}

}  // namespace

bool ptr_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

int check_ragged(int B, int T, int H_kv, int num_pages, int max_pages, int d, int dtype, int cache_format) {
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_INVALID_ARG;
  if (cache_format != FA_CACHE_16BIT && cache_format != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || H_kv < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // positions (of the rows past the last token of a tile too), table offsets and (page, head)
  // slabs are 32-bit inside the kernels
  if ((long long)max_pages * kPage + T >= (1ll << 31) - 256 || (long long)B * max_pages >= (1ll << 31) ||
      (long long)num_pages * H_kv >= (1ll << 31) || (long long)T * H_kv >= (1ll << 31))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

namespace {

// Checks of both entry points. k, v: the 16-bit side, `ks` / `vs` elements
// between tokens; `append`: the cache is the output.
int cache_impl(bool append, const void* k, const void* v, const void* kc, const void* vc, const void* ke,
               const void* ve, const int* table, const int* cu, const int* lens, int B, int T, int H_kv,
               int num_pages, int max_pages, int d, long long ks, long long vs, int dtype, int format,
               cudaStream_t strm) {
  int st = check_ragged(B, T, H_kv, num_pages, max_pages, d, dtype, format);
  if (st != FA_OK) return st;
  const long long width = (long long)H_kv * d;
  if (ks < width || vs < width || ks % 8 != 0 || vs % 8 != 0 || ks > (1ll << 40) || vs > (1ll << 40))
    return FA_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return FA_OK;   // nothing to write
  const bool fp8 = format == FA_CACHE_E4M3;
  if (!k || !v || !kc || !vc || !table || !cu || !lens) return FA_ERR_INVALID_ARG;
  if (fp8 ? (!ke || !ve) : (ke || ve)) return FA_ERR_INVALID_ARG;
  if (!ptr_aligned(k, 16) || !ptr_aligned(v, 16) || !ptr_aligned(kc, 16) || !ptr_aligned(vc, 16) ||
      !ptr_aligned(table, 4) || !ptr_aligned(cu, 4) || !ptr_aligned(lens, 4))
    return FA_ERR_INVALID_ARG;
  const size_t cache_rows = (size_t)num_pages * H_kv * kPage;
  const size_t cb = cache_rows * d * (fp8 ? 1 : 2), eb = fp8 ? cache_rows : 0;
  const void* ptr[9] = {k, v, kc, vc, ke, ve, table, cu, lens};
  const size_t len[9] = {((size_t)(T - 1) * ks + width) * 2, ((size_t)(T - 1) * vs + width) * 2, cb, cb, eb, eb,
                         (size_t)B * max_pages * 4, ((size_t)B + 1) * 4, (size_t)B * 4};
  // outputs: the cache and its exponents (2 .. 5), or k and v (0, 1)
  for (int i = append ? 2 : 0; i < (append ? 6 : 2); ++i)
    for (int j = 0; j < 9; ++j)
      if (i != j && ranges_overlap(ptr[i], len[i], ptr[j], len[j])) return FA_ERR_INVALID_ARG;
  st = check_current_device(ptr, 9);
  if (st != FA_OK) return st;
  CacheParams p{};
  p.r = Ragged{B, T, H_kv, num_pages, max_pages, cu, lens, table};
  p.k_in = p.k_out = static_cast<uint16_t*>(const_cast<void*>(k));
  p.v_in = p.v_out = static_cast<uint16_t*>(const_cast<void*>(v));
  p.k_stride = ks;
  p.v_stride = vs;
  p.k_cache = static_cast<uint8_t*>(const_cast<void*>(kc));
  p.v_cache = static_cast<uint8_t*>(const_cast<void*>(vc));
  p.k_exp = static_cast<uint8_t*>(const_cast<void*>(ke));
  p.v_exp = static_cast<uint8_t*>(const_cast<void*>(ve));
  const cudaError_t e = append ? launch_cache<false>(p, d, dtype, format, strm)
                               : launch_cache<true>(p, d, dtype, format, strm);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace fa

extern "C" int fa_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, unsigned char* k_exp,
                               unsigned char* v_exp, const int* block_table, const int* cu_seqlens,
                               const int* seqlens_k, int B, int T, int H_kv, int num_pages, int max_pages, int d,
                               long long k_stride, long long v_stride, int dtype, int cache_format,
                               void* stream) {
  return fa::cache_impl(true, k, v, k_cache, v_cache, k_exp, v_exp, block_table, cu_seqlens, seqlens_k, B, T, H_kv,
                        num_pages, max_pages, d, k_stride, v_stride, dtype, cache_format,
                        static_cast<cudaStream_t>(stream));
}

extern "C" int fa_cache_read(const void* k_cache, const void* v_cache, const unsigned char* k_exp,
                             const unsigned char* v_exp, const int* block_table, const int* cu_seqlens,
                             const int* seqlens_k, void* k, void* v, int B, int T, int H_kv, int num_pages,
                             int max_pages, int d, int dtype, int cache_format, void* stream) {
  const long long width = (long long)H_kv * d;
  return fa::cache_impl(false, k, v, k_cache, v_cache, k_exp, v_exp, block_table, cu_seqlens, seqlens_k, B, T,
                        H_kv, num_pages, max_pages, d, width, width, dtype, cache_format,
                        static_cast<cudaStream_t>(stream));
}
