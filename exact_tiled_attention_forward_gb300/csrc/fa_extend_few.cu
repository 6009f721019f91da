// fa_extend_paged for few rows: decode steps, where the rows that read one KV head
// (G query heads x up to max_q new tokens) number at most 16, the M of one mma.sync.
//
// Bound: HBM. The kernel streams every visible 128-key tile of K and V once per KV
// head, and everything else hides behind that stream.
//
// Split: the tiles of all (sequence, KV head) units form one line of W tiles in unit
// order, and CTA i of C takes tiles [i W / C, (i + 1) W / C): whatever the lengths,
// every CTA streams the same number of tiles, in one resident wave. Each CTA works
// its place in the line out itself from the lengths on the device (a scan over the
// sequences), so the host needs no lengths and a captured call follows the current
// ones. A unit inside one CTA's range is finished there; a unit that a range border
// cuts leaves FP32 partials (unnormalised O, running max and sum) in at most two
// slots per CTA, which fa_extend_few_merge_kernel combines.
//
// CTA: warp 4 streams tiles by TMA into a ring (unit borders do not stop it) and each
// unit's Q rows ahead of it; warps 0-3 each take 32 keys of every tile. On mma.sync
// m16n8k16, FP32 accumulation, keys and columns of V are the M of 16 and the query rows
// the N of 8 (one or two such groups, as the rows need): S^T = K Q^T, an online softmax
// over the warp's own keys, P^T turned into a B operand by movmatrix, O^T += V^T P^T. With
// the rows as M of 16, one token of four heads would leave three quarters of each product
// idle. The warps are merged in shared memory at the end of a unit.
//
// E4M3 caches: codes are widened to FP16 in registers (exact, one conversion per two
// codes). Q goes to FP16 times a power of two per row that puts the row's maximum in
// [2^14, 2^15): exact for all but elements 2^-29 below the maximum, which lose bits
// 2^-39 below it. A key's power of two multiplies its FP32 score (below 2^31 before: keys of up
// to 2^105 stay in range however small the query was). A value's goes into
// P, whose FP16 has no room for values of any size: a warp takes its keys of a tile in
// bands. A band is the keys that some row sees whose exponent is at most 12 below the largest
// one left, E; P' = 2^(s c - x) * 2^(ev - E + 14) with x the row's largest score in the band,
// so P' <= 2^14 and FP16 holds weights to 2^-27 of the band's largest, whatever weight or size
// other keys have. The band's products come out of the MMAs by themselves and are added
// to O in FP32 times 2^(x - m) 2^(E - 14); l takes its sum times 2^(x - m). Values within
// 2^12 of each other, the usual case, are one band and one pass.
//
// Measured (8 KV heads): one token of 16 sequences of 8192 keys, 4 heads a KV head, E4M3,
// d = 128, 52 us (271 MB at 5.2 TB/s, 77 % of a copy's rate), two tokens of 8 heads 70 us; one
// of 64 sequences, window 1024, FP16, d = 64, 38 us (132 MB at 3.5 TB/s: 1.7 units a CTA,
// so starting, borders and merging weigh as much).
#include "fa_serving.cuh"

#include <cmath>

namespace fa {
namespace {

constexpr int kFewThreads = 160;   // four consumer warps and the loading warp
constexpr int kFewConsumers = 128;
constexpr float kLn2x = 0.6931471805599453f;

template <int D, bool FP8, int NB>
struct FewCfg {
  static constexpr int kTileBytes = kPage * D * (FP8 ? 1 : 2);
  static constexpr int kExpBytes = FP8 ? kPage : 0;
  // CTAs per SM, all resident, and a CTA's ring of slots (one K or V tile each, 1024-byte
  // aligned; exponents of all slots follow). E4M3 tiles are half the bytes for the same
  // arithmetic and gain from a third CTA where 128 registers a thread suffice (one group of
  // query rows): 16 x 8192 keys, 4 heads, d = 128 / 64: 50.8 / 34.1 us with three, 52.4 / 33.8
  // with two; 16-bit 86.9 / 48.6 and 86.4 / 49.6
  static constexpr int kPerSm = FP8 && NB == 1 ? 3 : 2;
  static constexpr int kRing = (kPerSm == 3 ? 60 : 96) * 1024;
  static constexpr int kSlots = kRing / kTileBytes < 8 ? kRing / kTileBytes : 8;
  static constexpr int kOffExp = kSlots * kTileBytes;
  // the next unit's Q rows as they are, loaded ahead
  static constexpr int kOffRaw = kOffExp + kSlots * kExpBytes;
  // the four warps' O: [32 columns each][warp][row], and their (m, l)
  static constexpr int kOffBuf = kOffRaw + 8 * NB * D * 2;
  static constexpr int kOffMl = kOffBuf + 4 * 16 * 32 * 4;
  static constexpr int kOffBar = kOffMl + 4 * 16 * 2 * 4;
  static constexpr int kSmemBytes = kOffBar + (2 * kSlots + 2) * 8 + 1024;
  static_assert(kPerSm * (kSmemBytes + 64 + 1024) <= 228 * 1024, "CTAs per SM");
};

template <Elem E>
__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (E == Elem::F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2u(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Byte offset in a tile of 16-byte chunk `ch` of key row `key`, as TMA lays it out:
// 16-bit tiles in 64-column boxes with the 128-byte swizzle; E4M3 rows of 128 bytes
// with the 128-byte swizzle, of 64 bytes with the 64-byte swizzle.
template <int D, bool FP8>
__device__ __forceinline__ uint32_t tile_at(int key, int ch) {
  if constexpr (!FP8) return (uint32_t)((ch >> 3) * (kPage * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
  else if constexpr (D == 128) return (uint32_t)(key * 128 + ((ch ^ (key & 7)) << 4));
  else return (uint32_t)(key * 64 + ((ch ^ ((key >> 1) & 3)) << 4));
}

// Which of a group of 8 keys is row n of the score MMA. E4M3 rows of 128 bytes are read
// 16 bytes a lane, where the 8 lanes of a quarter warp hold rows (2i, 2i + 1) x 4 chunks:
// keys 4 apart put their chunks in different halves of the banks.
template <int D, bool FP8>
__device__ __forceinline__ int key_of_row(int n) {
  return FP8 && D == 128 ? ((n & 1) << 2) | (n >> 1) : n;
}

// Transposes an 8 x 8 block of 16-bit elements held as MMA fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t ld_shared_u8x(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// This CTA's stretch of the line of tiles, and the unit it starts in. (All counts are
// below 2^31: the host keeps B * H_kv * max_pages there.)
struct FewRange {
  int total;    // tiles of the line
  int s0, s1;   // tiles [s0, s1) of it
  int b, k;     // first unit: sequence b, the tile k of its H_kv * count tiles
};
// Where CTA i of n begins: i * total / n, without the product.
__device__ __forceinline__ int range_start(int total, int i, int n) {
  const int q = total / n, r = total - q * n;
  return q * i + r * i / n;   // n is a few hundred: r * i < n^2
}

__device__ __forceinline__ int tiles_of(const ExtendParams& p, int b) {
  const SeqTokens s = seq_tokens(p, b);
  if (s.n == 0) return 0;
  // (rows that see no key still get O = 0 and LSE = -inf: one fully masked tile)
  return max(key_tiles_of(s.p0, s.p0 + s.n, p.window, p.sinks, p.r.max_pages).count(), 1);
}

// The range of CTA i of n. Every warp works it out by itself, 128 sequences at a time
// (four a lane, their loads together): no barrier stands between the lengths and the
// first tile's load.
__device__ __forceinline__ FewRange few_range(const ExtendParams& p, int i, int n) {
  const int lane = threadIdx.x & 31;
  int first[4];   // tiles of the first 128 sequences
  int total = 0;
  for (int b0 = 0; b0 < p.r.B; b0 += 128) {
    int mine[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int b = b0 + 4 * lane + x;
      mine[x] = b < p.r.B ? tiles_of(p, b) * p.r.H_kv : 0;
    }
    if (b0 == 0) {
#pragma unroll
      for (int x = 0; x < 4; ++x) first[x] = mine[x];
    }
    total += __reduce_add_sync(0xffffffffu, mine[0] + mine[1] + mine[2] + mine[3]);
  }
  FewRange fr;
  fr.total = total;
  fr.s0 = range_start(total, i, n);
  fr.s1 = range_start(total, i + 1, n);
  fr.b = p.r.B;
  fr.k = 0;
  if (fr.s0 >= fr.s1) return fr;
  int before = 0;   // tiles of earlier sequences
  for (int b0 = 0; b0 < p.r.B; b0 += 128) {
    int mine[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int b = b0 + 4 * lane + x;
      mine[x] = b0 == 0 ? first[x] : b < p.r.B ? tiles_of(p, b) * p.r.H_kv : 0;
    }
    const int sum = mine[0] + mine[1] + mine[2] + mine[3];
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += up;
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    if (fr.s0 < before + all) {
      int lo = before + incl - sum;
      const unsigned who = __ballot_sync(0xffffffffu, fr.s0 >= lo && fr.s0 < lo + sum);
      int b = b0 + 4 * lane;
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (fr.s0 >= lo + mine[x]) {
          lo += mine[x];
          ++b;
        } else {
          break;
        }
      const int src = __ffs(who) - 1;
      fr.b = __shfl_sync(0xffffffffu, b, src);
      fr.k = __shfl_sync(0xffffffffu, fr.s0 - lo, src);
      break;
    }
    before += all;
  }
  return fr;
}

// A walk along the units of a range: (sequence, KV head), its tiles and how far into
// them this range goes.
struct FewUnit {
  int b, hk;
  SeqTokens s;
  KeyTiles kt;
  int count;        // tiles of the unit
  int k0, k1;       // this range's part of them
};
__device__ __forceinline__ void unit_load(const ExtendParams& p, FewUnit& u) {
  u.s = seq_tokens(p, u.b);
  u.kt = key_tiles_of(u.s.p0, u.s.p0 + u.s.n, p.window, p.sinks, p.r.max_pages);
  u.count = max(u.kt.count(), 1);
}
__device__ __forceinline__ void unit_first(const ExtendParams& p, const FewRange& fr, FewUnit& u) {
  u.b = fr.b;
  unit_load(p, u);
  u.hk = fr.k / u.count;
  u.k0 = fr.k - u.hk * u.count;
  u.k1 = min(u.count, u.k0 + (fr.s1 - fr.s0));
}
// The next unit, `left` tiles before the range's end (left > 0).
__device__ __forceinline__ void unit_next(const ExtendParams& p, FewUnit& u, int left) {
  if (++u.hk == p.r.H_kv) {
    u.hk = 0;
    do ++u.b;
    while (u.b + 1 < p.r.B && seq_tokens(p, u.b).n == 0);
    unit_load(p, u);
  }
  u.k0 = 0;
  u.k1 = min(u.count, left);
}

template <int D, Elem E, bool FP8, int NB>
__global__ void __launch_bounds__(kFewThreads, FewCfg<D, FP8, NB>::kPerSm)
    fa_extend_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const ExtendParams p) {
  using C = FewCfg<D, FP8, NB>;
  constexpr Elem M = FP8 ? Elem::F16 : E;   // type of the MMAs' operands
  // the scores are wanted again for a second band, which is rare: with 16 rows of 128 columns
  // their registers are needed before (16 x 8192 keys: 68 us, with them kept there 75)
  constexpr bool kPark = FP8 && NB == 2 && D == 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto full = [&](int s) -> uint32_t { return sb + C::kOffBar + 8 * s; };
  auto empty = [&](int s) -> uint32_t { return sb + C::kOffBar + 8 * (C::kSlots + s); };
  const uint32_t q_full = sb + C::kOffBar + 16 * C::kSlots, q_empty = q_full + 8;
  __shared__ int abort_word;
  volatile int* s_abort = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 4);
    abort_word = 0;
    fence_mbar_init();
  } else if (threadIdx.x == kFewConsumers) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  const FewRange fr = few_range(p, blockIdx.x, gridDim.x);
  __syncthreads();   // barriers are initialised
  // the merge kernel may be launched as SMs come free (it waits for this grid's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (fr.s0 >= fr.s1) {   // fewer tiles than CTAs: nothing here, and nothing for the merge
    if (threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (threadIdx.x < 16)
      __stcg(reinterpret_cast<float2*>(p.part_ml) + (size_t)blockIdx.x * 32 + threadIdx.x, make_float2(-INFINITY, 0.f));
    return;
  }
  FewUnit u;
  unit_first(p, fr, u);
  int left = fr.s1 - fr.s0;

  if (warp == 4) {
    // ======================= loads =======================
    if (lane == 0) {
      int it = 0, units = 0;   // tile loads issued (K and V alternate), units begun
      bool ok = true;
      for (;; ++units) {
        // the unit's query rows: a token's G heads lie together
        if (!mbar_wait(q_empty, ((uint32_t)units & 1u) ^ 1u, s_abort, p.status)) break;
        const uint32_t tok_bytes = (uint32_t)(p.G * D * 2);
        mbar_arrive_expect_tx(q_full, tok_bytes * (uint32_t)u.s.n);
        for (int t = 0; t < u.s.n; ++t)
          bulk_copy_1d(sb + C::kOffRaw + t * tok_bytes,
                       p.q + (size_t)(u.s.t0 + t) * p.q_stride + (size_t)u.hk * p.G * D, tok_bytes, q_full);
        int pg_next = page_at(p.r, u.b, u.kt.tile(u.k0));
        for (int k = u.k0; k < u.k1 && ok; ++k) {
          const int pg = pg_next;
          if (k + 1 < u.k1) pg_next = page_at(p.r, u.b, u.kt.tile(k + 1));   // on its way while slots are waited for
          // a page outside the cache: a slab past the end reads as zeros
          const int slab = pg >= 0 ? pg * p.r.H_kv + u.hk : p.r.num_pages * p.r.H_kv;
#pragma unroll
          for (int sel = 0; sel < 2; ++sel, ++it) {
            const int st = it % C::kSlots;
            if (!mbar_wait(empty(st), ((uint32_t)(it / C::kSlots) & 1u) ^ 1u, s_abort, p.status)) {
              ok = false;
              break;
            }
            const uint32_t dst = sb + st * C::kTileBytes;
            const void* tm = sel ? (const void*)&tmV : (const void*)&tmK;
            if constexpr (FP8) {
              const uint32_t de = sb + C::kOffExp + st * C::kExpBytes;
              if (pg < 0) {   // any factor will do for zeros
                for (int i = 0; i < C::kExpBytes; i += 16) st_shared_v4(de + i, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                fence_proxy_async_smem();
              }
              mbar_arrive_expect_tx(full(st), C::kTileBytes + (pg >= 0 ? C::kExpBytes : 0));
              if (pg >= 0) bulk_copy_1d(de, (sel ? p.v_exp : p.k_exp) + (size_t)slab * kPage, C::kExpBytes, full(st));
              tma_load_3d(dst, tm, full(st), 0, 0, slab);
            } else {
              mbar_arrive_expect_tx(full(st), C::kTileBytes);
#pragma unroll
              for (int bx = 0; bx < D / 64; ++bx)
                tma_load_3d(dst + bx * (kPage * 128), tm, full(st), bx * 64, 0, slab);
            }
          }
        }
        left -= u.k1 - u.k0;
        if (left <= 0 || !ok) {
          ++units;
          break;
        }
        unit_next(p, u, left);
      }
      // every load issued has landed before the CTA may exit
      volatile int never = 0;
      if (units > 0) mbar_wait(q_full, (uint32_t)(units - 1) & 1u, &never, p.status);
      for (int st = 0; st < C::kSlots; ++st) {
        const int n = it > st ? (it - st + C::kSlots - 1) / C::kSlots : 0;
        if (n > 0) mbar_wait(full(st), (uint32_t)(n - 1) & 1u, &never, p.status);
      }
    }
    return;
  }

  // ======================= four consumer warps =======================
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp * 32;   // this warp's keys of every tile
  // this lane's keys of a tile: key(mt, h) = kw + 16 mt + 8 h + kg, and its query rows:
  // row(nb, e) = 8 nb + 2 t + e
  const int kg = key_of_row<D, FP8>(g);
  int it = 0, units = 0;
  bool ok = true;
  for (;;) {
    const int R = u.s.n * p.G;
    // ---- Q^T as B operands (query row 8 nb + g, zero past R), and the rows' factors
    uint32_t qb[NB][D / 16][2];
    float crow[NB][2];   // scale log2(e), and the row's power of two undone
    if (ok) ok = mbar_wait_w(q_full, (uint32_t)units & 1u, s_abort, p.status);
    ++units;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int m = 8 * nb + g;
      const uint32_t row = sb + C::kOffRaw + (uint32_t)m * (D * 2);   // token m / G, head m % G
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        uint2 x = make_uint2(0, 0);
        if (m < R) {
          // E4M3: lane t holds elements (t + 4 i) * 16 + 4 j + {0, 1 | 2, 3} of K-step (i, j),
          // the order in which its K codes lie
          if constexpr (FP8) x = ld_shared_v2u(row + ((t + 4 * (s >> 2)) * 16 + 4 * (s & 3)) * 2);
          else x = make_uint2(ld_shared_u32(row + (s * 8 + t) * 4), ld_shared_u32(row + (s * 8 + 4 + t) * 4));
        }
        qb[nb][s][0] = x.x;
        qb[nb][s][1] = x.y;
      }
      float cg = p.c;
      if constexpr (FP8 && E != Elem::F16) {
        uint32_t top = 0;   // the row's largest magnitude, as a BF16 pattern
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t v = qb[nb][s][x] & 0x7FFF7FFFu;
            top = max(top, max(v & 0xFFFFu, v >> 16));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int xb = (int)(top >> 7);   // its biased exponent; 255: infinity or NaN
        const int sh = xb == 255 ? 0 : min(127 + 14 - xb, 120);
        const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
        cg = p.c * __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t v = qb[nb][s][x];
            qb[nb][s][x] = pack_f16x2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) crow[nb][e] = __shfl_sync(0xffffffffu, cg, (2 * t + e) * 4);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty);

    // the tiles that some row sees only in part: positions of the unit's first and last token
    const int pos_lo = u.s.p0, pos_hi = u.s.p0 + u.s.n - 1;
    float mrow[NB][2], lrow[NB][2];
    float oacc[D / 16][NB][4];   // O^T: 16 columns by 8 rows each
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      mrow[nb][0] = mrow[nb][1] = -INFINITY;
      lrow[nb][0] = lrow[nb][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[i][nb][e] = 0.f;
    }

    for (int k = u.k0; k < u.k1; ++k) {
      const int key0 = u.kt.tile(k) * kPage;
      const int stK = it % C::kSlots;
      const uint32_t phK = (uint32_t)(it / C::kSlots) & 1u;
      ++it;
      const int stV = it % C::kSlots;
      const uint32_t phV = (uint32_t)(it / C::kSlots) & 1u;
      ++it;
      if (ok) ok = mbar_wait_w(full(stK), phK, s_abort, p.status);
      if (!ok) continue;   // a wait gave up: only the barriers below are still taken
      // ---- S^T = K Q^T for this warp's 32 keys: two blocks of 16
      const uint32_t tk = sb + stK * C::kTileBytes;
      float sacc[NB][2][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sacc[nb][mt][e] = 0.f;
      if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint4 w4[2][2];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) w4[mt][h] = ld_shared_v4u(tk + tile_at<D, FP8>(kw + 16 * mt + 8 * h + kg, t + 4 * i));
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t a[4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4& w = w4[mt][h];
                e4m3x4_to_f16x2x2(j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w, a[h], a[2 + h]);
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_16816<M>(sacc[nb][mt], a, qb[nb][4 * i + j][0], qb[nb][4 * i + j][1]);
            }
        }
      } else {
        const int i = lane >> 3, rr = lane & 7;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            uint32_t a[4];
            ldmatrix_x4(tk + tile_at<D, FP8>(kw + 16 * mt + 8 * (i & 1) + rr, 2 * s + (i >> 1)), a);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma_16816<M>(sacc[nb][mt], a, qb[nb][s][0], qb[nb][s][1]);
          }
      }
      // ---- E4M3: a key's power of two on its scores
      if constexpr (FP8) {
        const uint32_t ek = sb + C::kOffExp + stK * C::kExpBytes + kw + kg;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // exp_factor, but infinite for a NaN row, whose codes are NaN
            const float f = __uint_as_float(max(ld_shared_u8x(ek + 16 * mt + 8 * h) << 23, 0x00400000u));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              sacc[nb][mt][2 * h] *= f;
              sacc[nb][mt][2 * h + 1] *= f;
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(stK));
      const int left_keys = u.s.len - key0;   // keys of the tile that exist (a mask cuts the rest)
      const uint32_t tv = sb + stV * C::kTileBytes;
      // ---- the mask: key (relative to the tile) is seen iff key < hi and (key >= lo or key < snk)
      // (tokens past the table see none of any tile)
      const int snk = p.sinks - key0;
      const bool cut = key0 + kPage - 1 > pos_lo || pos_hi >= p.r.max_pages * kPage ||
                       (p.window > 0 && key0 <= pos_hi - p.window && snk < kPage);
      if (cut) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // position of the row; below every key for rows past R or the table
            const int r = 8 * nb + 2 * t + e;
            int pos = r < R ? pos_lo + r / p.G : -1;
            if (pos >= p.r.max_pages * kPage) pos = -1;
            const int hi = pos + 1 - key0;
            const int lo = p.window > 0 ? hi - p.window : -kPage;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = kw + 16 * mt + 8 * h + kg;
                if (!(key < hi && (key >= lo || key < snk))) sacc[nb][mt][2 * h + e] = -INFINITY;
              }
          }
      }
      // V rows past the sequence's end may hold anything, NaN included, and 0 * NaN is
      // NaN: zero them (each warp its own keys)
      auto zero_past_end = [&] {
        if (left_keys >= kPage) return;
        constexpr int kCh = D * (FP8 ? 1 : 2) / 16;
        for (int i = lane; i < 32 * kCh; i += 32) {
          const int key = kw + i / kCh;
          if (key >= left_keys) st_shared_v4(tv + tile_at<D, FP8>(key, i % kCh), 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();   // before the slot's next TMA load
        __syncwarp();
      };
      // E4M3: V's exponent bytes plus 1; 0 for keys of a band before, and for keys that no row of
      // the unit sees (a row's window begins no earlier than the first one's), which must
      // not shift the others
      [[maybe_unused]] uint32_t vb[2][2] = {};
      if constexpr (FP8) {
        ok = mbar_wait_w(full(stV), phV, s_abort, p.status);
        if (!ok) continue;
        const uint32_t ev = sb + C::kOffExp + stV * C::kExpBytes + kw + kg;
        const int hi = pos_hi + 1 - key0, lo = p.window > 0 ? pos_lo + 1 - key0 - p.window : -kPage;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = kw + 16 * mt + 8 * h + kg;
            vb[mt][h] = key < hi && (key >= lo || key < snk) ? ld_shared_u8x(ev + 16 * mt + 8 * h) + 1 : 0u;
          }
        zero_past_end();
      }
      // ---- online softmax over this warp's keys, and O^T += V^T P^T; E4M3: band by band
      for (;;) {
        [[maybe_unused]] uint32_t top = 0, least = 0;   // E4M3: E + 1, and the band's lowest
        if constexpr (FP8) {
          top = __reduce_max_sync(0xffffffffu, max(max(vb[0][0], vb[0][1]), max(vb[1][0], vb[1][1])));
          if (top == 0) break;
          least = top > 12 ? top - 12 : 1;
          if constexpr (kPark) {   // the scores wait in the buffers of the unit's end, idle by now
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
                st_shared_v4(sb + C::kOffBuf + ((nb * 2 + mt) * kFewConsumers + threadIdx.x) * 16, __float_as_uint(sacc[nb][mt][0]),
                             __float_as_uint(sacc[nb][mt][1]), __float_as_uint(sacc[nb][mt][2]), __float_as_uint(sacc[nb][mt][3]));
          }
        }
        auto in_band = [&](int mt, int h) { return !FP8 || vb[mt][h] >= least; };
        float mx[NB][2];
        [[maybe_unused]] float xb[NB][2];   // E4M3: the band's largest score of each row
        bool up = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (in_band(mt, h)) x = fmaxf(x, sacc[nb][mt][2 * h + e]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x *= crow[nb][e];   // (-inf stays -inf: crow > 0)
            if constexpr (FP8) xb[nb][e] = x;
            mx[nb][e] = fmaxf(mrow[nb][e], x);
            up |= mx[nb][e] > mrow[nb][e];
          }
        // O is touched only where a maximum rose in some row
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (0 from -inf: nothing was summed yet)
              const float alpha = mx[nb][e] > mrow[nb][e] ? ex2_approx(mrow[nb][e] - mx[nb][e]) : 1.f;
              mrow[nb][e] = mx[nb][e];
              lrow[nb][e] *= alpha;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                oacc[i][nb][e] *= alpha;
                oacc[i][nb][2 + e] *= alpha;
              }
            }
        }
        uint32_t pb[2][NB][2];   // P^T as B operands: keys 16 mt + 8 h .., rows 8 nb ..
        [[maybe_unused]] float gain[NB][2];   // E4M3: what the band's products count for in O
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float ref[2], sum[2] = {0.f, 0.f};   // what the scores are held against, and their sum
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ref[e] = FP8 ? xb[nb][e] : mrow[nb][e];
            if (ref[e] == -INFINITY) ref[e] = 0.f;
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                x[e] = in_band(mt, h) ? ex2_approx(fmaf(sacc[nb][mt][2 * h + e], crow[nb][e], -ref[e])) : 0.f;
                if constexpr (FP8) sum[e] += x[e];
                else lrow[nb][e] += x[e];   // this lane's keys; the eight lanes of a row are added at the end
              }
              if constexpr (FP8) {   // 2^(14 + byte - E)
                const float f = in_band(mt, h) ? __uint_as_float((141u + vb[mt][h] - top) << 23) : 0.f;
                x[0] *= f;
                x[1] *= f;
              }
              pb[mt][nb][h] = transpose8(pack2<M>(x[0], x[1]));
            }
          if constexpr (FP8)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = xb[nb][e] == -INFINITY ? 0.f : ex2_approx(xb[nb][e] - mrow[nb][e]);
              lrow[nb][e] += sum[e] * f;   // (a NaN among the band's scores makes its sum one)
              // O is held times 2^8, so that 2^(E - 14) stays a normal number down to the
              // smallest byte that fa_cache_append writes (top = 8)
              gain[nb][e] = f * __uint_as_float(top > 7 ? (top - 7) << 23 : 0x00400000u >> (7 - top));
            }
        }
        if constexpr (!FP8) {
          ok = mbar_wait_w(full(stV), phV, s_abort, p.status);
          if (!ok) break;
          zero_past_end();
        }
        // ---- O^T += V^T P^T
        const int i = lane >> 3, rr = lane & 7;
        if constexpr (FP8) {
#pragma unroll
          for (int dp = 0; dp < D / 32; ++dp) {
            // 8 x 8 blocks of code pairs, transposed: a lane gets two keys' codes of two
            // adjacent columns; the bytes sorted by column are rows g (even columns of the
            // 16) and g + 8 (odd ones) of an A operand
            uint32_t av[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
              ldmatrix_x4_t(tv + tile_at<D, FP8>(kw + 16 * mt + 8 * (i & 1) + key_of_row<D, FP8>(rr), 2 * dp + (i >> 1)), av[mt]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float acc[NB][4];   // the band's own products
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nb][e] = 0.f;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                uint32_t a[4];
                e4m3x4_to_f16x2x2(__byte_perm(av[mt][2 * x], 0, 0x3120), a[0], a[1]);
                e4m3x4_to_f16x2x2(__byte_perm(av[mt][2 * x + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_16816<M>(acc[nb], a, pb[mt][nb][0], pb[mt][nb][1]);
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  oacc[2 * dp + x][nb][e] = fmaf(acc[nb][e], gain[nb][e & 1], oacc[2 * dp + x][nb][e]);
            }
          }
          bool rest = false;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (in_band(mt, h)) vb[mt][h] = 0;
              rest |= vb[mt][h] != 0;
            }
          if (!__any_sync(0xffffffffu, rest)) break;
          if constexpr (kPark) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                const float4 w = ld_shared_v4f(sb + C::kOffBuf + ((nb * 2 + mt) * kFewConsumers + threadIdx.x) * 16);
                sacc[nb][mt][0] = w.x; sacc[nb][mt][1] = w.y; sacc[nb][mt][2] = w.z; sacc[nb][mt][3] = w.w;
              }
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
              uint32_t av[4];
              ldmatrix_x4_t(tv + tile_at<D, FP8>(kw + 16 * mt + 8 * (i >> 1) + rr, 2 * dp + (i & 1)), av);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma_16816<M>(oacc[dp][nb], av, pb[mt][nb][0], pb[mt][nb][1]);
            }
          break;
        }
      }
      if (!ok) continue;
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(stV));
    }

    // ---- the four warps' (m, l, O) of this unit into one
    const uint32_t mls = sb + C::kOffMl;   // [warp][row] (m, l)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) lrow[nb][e] += __shfl_xor_sync(0xffffffffu, lrow[nb][e], off);
        if (g == 0)
          st_shared_v2(mls + (warp * 16 + 8 * nb + 2 * t + e) * 8, __float_as_uint(mrow[nb][e]), __float_as_uint(lrow[nb][e]));
      }
    const bool all_ok = named_bar_and(1, kFewConsumers, ok);
    constexpr float back = FP8 ? 1.f / 256.f : 1.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 ml = ld_shared_v2f(mls + (x * 16 + 8 * nb + 2 * t + e) * 8);
          if (ml.y != 0.f) top = fmaxf(top, ml.x);
        }
        const bool any = lrow[nb][e] != 0.f;   // else this warp saw no key of the row (a NaN sum is one)
        const float wt = ex2_approx(mrow[nb][e] - top) * back;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          oacc[i][nb][e] = any ? oacc[i][nb][e] * wt : 0.f;
          oacc[i][nb][2 + e] = any ? oacc[i][nb][2 + e] * wt : 0.f;
        }
      }
    const bool whole = u.k0 == 0 && u.k1 == u.count;
    const int slot = 2 * blockIdx.x + (u.k0 == 0 ? 1 : 0);   // a unit cut at its end: slot 1; one that goes on: slot 0
    // the warps' O side by side in shared memory, 32 columns at a time, as many at once as
    // the rows leave room for (one barrier before their sums and one after). A row's 16-byte
    // chunks are XORed with the row against bank conflicts.
    const int at_once = R <= 4 ? 4 : R <= 8 ? 2 : 1;
    const uint32_t bufs = sb + C::kOffBuf;
    auto place = [&](int blk, int w, int m, int c4) {   // chunk c4 of row m of warp w
      return bufs + (uint32_t)((((blk * 4 + w) * (16 / at_once) + m) * 8 + (c4 ^ (m & 7))) * 16);
    };
#pragma unroll
    for (int h = 0; h < D / 32; ++h) {
      const int blk = h & (at_once - 1);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int m = 8 * nb + 2 * t + e;
          if (m >= R) continue;
#pragma unroll
          for (int c = 0; c < 2; ++c) {   // 16 columns
            const float* a = oacc[2 * h + c][nb];
            if constexpr (FP8) {          // even columns in the upper rows of the accumulator, odd ones in the lower
              st_shared_v2(place(blk, warp, m, 4 * c + (g >> 1)) + (g & 1) * 8, __float_as_uint(a[e]), __float_as_uint(a[2 + e]));
            } else {
              st_shared_u32(place(blk, warp, m, 4 * c + (g >> 2)) + (g & 3) * 4, __float_as_uint(a[e]));
              st_shared_u32(place(blk, warp, m, 4 * c + 2 + (g >> 2)) + (g & 3) * 4, __float_as_uint(a[2 + e]));
            }
          }
        }
      if (blk != at_once - 1 && h != D / 32 - 1) continue;
      named_bar_sync(1, kFewConsumers);
      // out: eight columns a thread, of the blk + 1 blocks gathered
      const int per_row = (blk + 1) * 4;
      if (all_ok)
        for (int idx = threadIdx.x; idx < R * per_row; idx += kFewConsumers) {
          const int m = idx / per_row, c8 = idx - m * per_row;   // 8-column chunk of the gathered blocks
          float top = -INFINITY, L = 0.f;
          float2 wl[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            wl[x] = ld_shared_v2f(mls + (x * 16 + m) * 8);
            if (wl[x].y != 0.f) top = fmaxf(top, wl[x].x);
          }
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (wl[x].y != 0.f) L += ex2_approx(wl[x].x - top) * wl[x].y;
            const float4 a = ld_shared_v4f(place(c8 >> 2, x, m, (2 * c8) & 7));
            const float4 b = ld_shared_v4f(place(c8 >> 2, x, m, ((2 * c8) & 7) + 1));
            o[0] += a.x; o[1] += a.y; o[2] += a.z; o[3] += a.w;
            o[4] += b.x; o[5] += b.y; o[6] += b.z; o[7] += b.w;
          }
          const int col = (h - blk) * 32 + c8 * 8;
          if (whole) {
            const int tok = m / p.G;
            const size_t orow = (size_t)(u.s.t0 + tok) * p.H_q + u.hk * p.G + (m - tok * p.G);
            if (!FA_DBG_OK(p.status, orow < (size_t)p.r.T * p.H_q && col + 8 <= D)) continue;
            const float inv = L != 0.f ? 1.f / L : 0.f;
            st_global_v4(static_cast<uint16_t*>(p.o) + orow * D + col, pack2<E>(o[0] * inv, o[1] * inv),
                         pack2<E>(o[2] * inv, o[3] * inv), pack2<E>(o[4] * inv, o[5] * inv),
                         pack2<E>(o[6] * inv, o[7] * inv));
            if (col == 0 && p.lse) p.lse[orow] = L != 0.f ? (top + __log2f(L)) * kLn2x : -INFINITY;
          } else if (FA_DBG_OK(p.status, slot < 2 * (int)gridDim.x && m < 16)) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + ((size_t)slot * 16 + m) * D + col);
            __stcg(dst, make_float4(o[0], o[1], o[2], o[3]));
            __stcg(dst + 1, make_float4(o[4], o[5], o[6], o[7]));
            if (col == 0)
              __stcg(reinterpret_cast<float2*>(p.part_ml) + (size_t)slot * 16 + m, make_float2(L != 0.f ? top : -INFINITY, L));
          }
        }
      named_bar_sync(1, kFewConsumers);   // the buffers (and at the end the (m, l)) are free
    }
    left -= u.k1 - u.k0;
    if (left <= 0) {
      // the range's last unit: for the merge, whether it begins here and goes on past the
      // range (rows n > 0), and in which CTA it ends
      if (threadIdx.x == 0) {
        const bool cut = u.k0 == 0 && u.k1 < u.count;
        // the unit ends in the first CTA whose range reaches its last tile
        const int end = fr.s1 + (u.count - u.k1), n = (int)gridDim.x;
        int last = blockIdx.x;
        for (int step = 256; step > 0; step >>= 1)   // (n < 512)
          if (last + step < n && range_start(fr.total, last + step, n) < end) last += step;
        p.cuts[blockIdx.x] = make_int4(cut ? u.s.n * p.G : 0, u.s.t0, u.hk, last);
      }
      break;
    }
    unit_next(p, u, left);
  }
}

// Combines the partials of the units that range borders cut: block (i, m) looks up
// whether a unit begins in CTA i's range and ends past it; if so, row m of the unit is
// M = max m_x, L = sum 2^(m_x - M) l_x, O = sum 2^(m_x - M) O_x / L over slot 1 of CTA i and
// slot 0 of the CTAs after it up to the unit's last. Four groups of threads share the
// parts, each with four columns a thread, so that their loads are in flight together.
constexpr int kMergeMax = 512;   // parts: CTAs of a launch at most
template <int D, Elem E>
__global__ void __launch_bounds__(D) fa_extend_few_merge_kernel(const ExtendParams p, const int ctas) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float wt[kMergeMax];
  __shared__ float4 sum[4][D / 4];
  __shared__ float red[D / 32];
  const int i = blockIdx.x, m = blockIdx.y, tid = threadIdx.x;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  auto slot = [&](int x) { return (size_t)(x == 0 ? 2 * i + 1 : 2 * (i + x)) * 16 + m; };
  constexpr int kCh = D / 4;   // 16-byte chunks of a row: one thread each, in four groups
  const int grp = tid / kCh, ch = tid - grp * kCh;
  // what most blocks need goes out together: the entry, and each group's first part
  const bool there = i + grp < ctas;
  const float4 o_first = there ? __ldcg(reinterpret_cast<const float4*>(p.part_o + slot(grp) * D) + ch)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
  const float2 ml_first = i + tid < ctas ? __ldcg(ml + slot(tid)) : make_float2(-INFINITY, 0.f);
  const int4 cut = __ldcg(p.cuts + i);
  if (m >= cut.x) return;
  const int parts = min(cut.w, ctas - 1) - i + 1;
  float M = tid < parts && ml_first.y != 0.f ? ml_first.x : -INFINITY;
  for (int x = tid + D; x < parts; x += D) {
    const float2 v = __ldcg(ml + slot(x));
    if (v.y != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if ((tid & 31) == 0) red[tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < D / 32; ++w) M = fmaxf(M, red[w]);
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  {
    for (int x = tid; x < parts; x += D) {
      const float2 v = x == tid ? ml_first : __ldcg(ml + slot(x));
      const float w = v.y != 0.f ? ex2_approx(v.x - M) : 0.f;
      wt[x] = w;
      L += w * v.y;
    }
    __syncthreads();
#pragma unroll 4
    for (int x = grp; x < parts; x += 4) {
      const float w = wt[x];
      // (a part that saw no key, weight 0, may have left its O unwritten)
      const float4 o = w == 0.f   ? make_float4(0.f, 0.f, 0.f, 0.f)
                       : x == grp ? o_first
                                  : __ldcg(reinterpret_cast<const float4*>(p.part_o + slot(x) * D) + ch);
      acc.x += w * o.x; acc.y += w * o.y; acc.z += w * o.z; acc.w += w * o.w;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = L;
  sum[grp][ch] = acc;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) L += red[w];
  const int tok = m / p.G;
  const size_t orow = (size_t)(cut.y + tok) * p.H_q + cut.z * p.G + (m - tok * p.G);
  if (!FA_DBG_OK(p.status, orow < (size_t)p.r.T * p.H_q)) return;
  if (tid < kCh) {
    const float inv = L != 0.f ? 1.f / L : 0.f;
    float4 a = sum[0][tid];
#pragma unroll
    for (int g = 1; g < 4; ++g) {
      const float4 b = sum[g][tid];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    uint2 out;
    out.x = pack2<E>(a.x * inv, a.y * inv);
    out.y = pack2<E>(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + orow * D + 4 * tid) = out;
  }
  if (tid == 0 && p.lse) p.lse[orow] = L != 0.f ? (M + __log2f(L)) * kLn2x : -INFINITY;
}

template <int D, Elem E, bool FP8, int NB>
cudaError_t launch_few_t(const CUtensorMap& tk, const CUtensorMap& tv, const ExtendParams& p, cudaStream_t stream) {
  using C = FewCfg<D, FP8, NB>;
  static bool attr[64] = {false};   // per device; a repeated set is harmless
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!attr[dev]) {
    cudaError_t e = cudaFuncSetAttribute(fa_extend_few_kernel<D, E, FP8, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  const int ctas = few_ctas(FP8, NB);
  cudaError_t e = launch_kernel(fa_extend_few_kernel<D, E, FP8, NB>, dim3((unsigned)ctas), dim3(kFewThreads), C::kSmemBytes,
                                stream, tk, tv, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)(p.G * p.max_q));
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_extend_few_merge_kernel<D, E>, p, ctas);
}

}  // namespace

int few_ctas(bool fp8, int groups) {
  const int per_sm = fp8 && groups == 1 ? FewCfg<128, true, 1>::kPerSm : FewCfg<128, false, 1>::kPerSm;
  const int n = per_sm * num_sms();
  return n < kMergeMax ? n : kMergeMax;
}

cudaError_t launch_extend_few(int d, int dtype, int format, const CUtensorMap& tk, const CUtensorMap& tv,
                              const ExtendParams& p, cudaStream_t stream) {
  const bool fp8 = format == FA_CACHE_E4M3, one = few_groups(p) == 1;
#define FA_FEW_GO(DD, EE)                                                                                        \
  return fp8 ? (one ? launch_few_t<DD, EE, true, 1>(tk, tv, p, stream) : launch_few_t<DD, EE, true, 2>(tk, tv, p, stream)) \
             : (one ? launch_few_t<DD, EE, false, 1>(tk, tv, p, stream) : launch_few_t<DD, EE, false, 2>(tk, tv, p, stream))
  if (dtype == FA_DTYPE_FP16) {
    if (d == 128) FA_FEW_GO(128, Elem::F16);
    FA_FEW_GO(64, Elem::F16);
  }
  if (d == 128) FA_FEW_GO(128, Elem::BF16);
  FA_FEW_GO(64, Elem::BF16);
#undef FA_FEW_GO
}

}  // namespace fa
