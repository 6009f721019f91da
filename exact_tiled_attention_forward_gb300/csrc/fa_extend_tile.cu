// Attention of many rows over a paged cache (fa_extend_paged) or over contiguous K and V
// (fa_forward_window): tcgen05 tiles of packed query rows, causal, with an optional
// sliding window and sinks.
//
// Rows: a 128-row tile holds TQ = 128 / G consecutive tokens of one sequence times the G
// query heads that read one KV head (row = token * G + head), so each K/V tile is loaded
// once for the whole group and a chunk of a few tokens still fills a tile. A work unit is
// two such tiles (2 TQ tokens) of one (sequence, KV head): its key tiles are those its
// tokens see (the sink tiles, then the window's), in order.
//
// Items: a unit's key range, cut into s parts when that shortens the whole (few units,
// long keys). Every CTA works the plan out itself from the lengths on the device: it
// weighs up to 16 cuts and takes the one with the least estimated time. The grid has a CTA
// for every item there can be; one CTA stays on each SM and takes over the CTAs that have
// not been launched yet (cluster launch control), so items go to whichever SM is free,
// longest first, without a counter in memory. A sequence's items come in groups of KV
// heads whose K and V fit in half of L2 together. Parts leave unnormalised FP32
// partials, combined by fa_extend_tile_merge_kernel.
//
// CTA (384 threads), tensor memory and the softmax are those of fa_fwd_kernel (its file
// explains them): two ping-pong query tiles, warpgroups 0 and 1 one query row a thread,
// warp 8 loads, warp 9 issues MMAs; S(j + 1) of a tile is issued right behind P V(j).
// Across items nothing drains: the loading thread works out the next item (in shared
// memory, for every role), its loads run ahead, and its first S overlaps this one's
// epilogue. Rows past the last token load whatever follows and are not stored.
//
// E4M3 caches: codes are loaded into a ring of their own, and a fourth warpgroup widens
// them to 16-bit tiles (exactly, the row's power of two multiplied in), so the MMAs see
// what a 16-bit cache of these values would hold. Two widening warps in the third
// warpgroup's idle slots kept the 384-thread register split but set the pace (2 x 2048
// tokens, window 4096: 458 us; with the arithmetic left out 354, a 16-bit cache 300).
//
// Bound: the tensor cores over 16-bit caches; over E4M3 ones shared memory, which the codes
// pass through twice more. Measured (32/8 heads, d = 128, BF16): 4096 new tokens of 32768
// 1446 us (1425 TFLOP/s), 4 x 512 of 8192 163 us (1100), E4M3 2 x 2048, window 4096, 338 us
// (790); fa_forward_window, N = 8192, window 1024, 145 us (890 over the pairs that see each
// other, 20 % of the tiles' work lies outside).
#include "fa_fwd_kernel.cuh"
#include "fa_serving.cuh"

namespace fa {
namespace {

template <int D, bool FP8>
struct TCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = 128 * 128;          // 128 rows x 64 16-bit columns
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStages = (FP8 ? 3 : 4) * (D == 128 ? 1 : 2);
  static constexpr int kRawBytes = FP8 ? 128 * D : 0;  // a tile of codes
  static constexpr int kRaw = FP8 ? (D == 128 ? 3 : 6) : 0;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffRaw = kOffKV + kStages * kTileBytes;
  static constexpr int kOffExp = kOffRaw + kRaw * kRawBytes;
  // epilogue staging: 32 rows of kStgCols 16-bit columns for each softmax warp
  static constexpr int kStgCols = FP8 && D == 128 ? 16 : 32;
  static constexpr int kStgBytes = 32 * kStgCols * 2;
  static constexpr int kOffStg = kOffExp + kRaw * 128;
  static constexpr int kOffPlan = kOffStg + 8 * kStgBytes;
  // plan: item prefix (+ 1), blocks and parts of every sequence
  static constexpr int kOffBar = kOffPlan + ((kTileMaxSeqs * 3 + 4) * 4);
  static constexpr int kBarQ = 0, kBarQFree = 1, kBarFull = 2, kBarEmpty = kBarFull + kStages,
                       kBarS = kBarEmpty + kStages, kBarP1 = kBarS + 2, kBarP2 = kBarP1 + 2, kBarO = kBarP2 + 2,
                       kBarDrain = kBarO + 2, kBarRawFull = kBarDrain + 1, kBarRawEmpty = kBarRawFull + kRaw,
                       kBarItem = kBarRawEmpty + kRaw, kBarItemFree = kBarItem + 2, kBarNext = kBarItemFree + 2,
                       kNumBars = kBarNext + 1;
  // answer to a request for the next CTA (16 bytes), two item slots, TMEM address and abort flag
  static constexpr int kOffNext = (kOffBar + kNumBars * 8 + 15) & ~15;
  static constexpr int kOffItem = kOffNext + 16;
  static constexpr int kOffMisc = kOffItem + 2 * 64;
  static constexpr int kItemReaders = FP8 ? 13 : 9;   // warps: MMA, 8 softmax, 4 widening
  // threads, and registers a thread after the split: 384 x 168 = 128 x (216 + 216 + 72)
  // or 512 x 128 = 128 x (200 + 200 + 56 + 56)
  static constexpr int kThreadsT = FP8 ? 512 : 384;
  static constexpr int kRegsSoft = FP8 ? 200 : 216, kRegsRest = FP8 ? 56 : 72;
  static constexpr int kSmemUsed = kOffMisc + 16 + 1024;
  static constexpr int kSmemBytes = kSmemUsed > 120 * 1024 ? kSmemUsed : 120 * 1024;   // one CTA per SM (tensor memory)
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static_assert(kOffBar % 8 == 0, "barriers are 8-byte aligned");
  __device__ static constexpr uint32_t tm_s(int X) { return X ? 128u : 0u; }
  __device__ static constexpr uint32_t tm_o(int X) { return X ? 384u : 256u; }
};

// How far a row's reference max may lag its true max (log2 units). BF16 has FP32's
// range, so P up to 2^48 costs neither precision (its 8 bits are relative) nor range: sums
// over 2^20 keys of values up to 2^59 still fit FP32. A reference from the row's first
// live tile then almost always lasts. Scores spread over 40 units (one key in a hundred
// eight times larger), 4 x 512 tokens over 8192 keys: 192 us with fa_fwd_kernel's 16, 173
// with 32, 167 with 48. FP16's P ends at 2^15, as there.
template <Elem E>
struct TileLag {
  static constexpr float kTau = E == Elem::F16 ? Lag<E>::kTau : 48.0f;
  static constexpr float kSumCap = E == Elem::F16 ? Lag<E>::kSumCap : 281474976710656.0f;   // 2^48
};

// The plan in shared memory, and what it amounts to.
struct TilePlan {
  int* prefix;    // [B + 1] items before each sequence (prefix[B]: all)
  int* blocks;    // [B] units per KV head
  int* parts;     // [B] parts of each unit's key range
  int items;
  int longest;    // tiles of the longest part; 0: nothing is cut
};

__device__ __forceinline__ SeqTokens tile_seq(const TileParams& p, int b) {
  if (p.e.r.table) return seq_tokens(p.e, b);
  return SeqTokens{0, p.N_q, p.N_k - p.N_q, p.N_k};
}

// Called by all NT threads; `red`: 20 words of shared memory. In whole numbers
// throughout, so that every CTA agrees. given: 0, or the longest part of a plan made before
// (the merge kernel follows the one its main kernel wrote down).
template <int NT>
__device__ __forceinline__ TilePlan tile_plan(const TileParams& p, int* mem, unsigned long long* red, int given = 0) {
  const int B = p.e.r.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  TilePlan pl{mem, mem + kTileMaxSeqs + 1, mem + 2 * kTileMaxSeqs + 1, 0, 0};
  const int U = 2 * p.TQ;
  if (tid < 20) red[tid] = 0;
  __syncthreads();
  // per sequence: units, and the tiles of its longest; overall: the longest, and twice the work
  int top = 0;
  unsigned long long work = 0;
  for (int b = tid; b < B; b += NT) {
    const SeqTokens s = tile_seq(p, b);
    const int nb = (s.n + U - 1) / U;
    int tmax = 0;
    if (nb > 0) {
      const int last = key_tiles_of(s.p0 + (nb - 1) * U, s.p0 + s.n, p.e.window, p.e.sinks, p.key_tiles).count();
      const int first = key_tiles_of(s.p0, s.p0 + min(U, s.n), p.e.window, p.e.sinks, p.key_tiles).count();
      // (under a window the blocks between may have one tile more than either)
      tmax = max(max(first, last) + (p.e.window > 0 && nb > 2 ? 1 : 0), 1);
      work += (unsigned long long)nb * (unsigned long long)(first + last);
    }
    pl.blocks[b] = nb;
    pl.parts[b] = tmax;
    top = max(top, tmax);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    work += __shfl_xor_sync(0xffffffffu, work, off);
  }
  if (lane == 0) {
    atomicMax(red + 16, (unsigned long long)top);
    atomicAdd(red + 17, work);
  }
  __syncthreads();
  top = max((int)red[16], 1);
  int best = 0;
  if (given == 0 && p.max_split_items > 0 && top > 1) {
    // items of each candidate cut c (lane c of every warp; a warp takes every NT / 32-th
    // sequence): parts of at most X = ceil(top / (c + 1)) tiles
    const int Xc = (top + (lane & 15)) / ((lane & 15) + 1);
    long long cnt = 0;
    for (int b = warp; b < B; b += NT / 32) cnt += (long long)pl.blocks[b] * ((pl.parts[b] + Xc - 1) / Xc);
    if (lane < 16 && cnt) atomicAdd(red + lane, (unsigned long long)cnt);
    __syncthreads();
    // time in key-tile steps of one CTA (here times 2 SMs): an even share of the work plus
    // half an item (the last wave's raggedness), or one item where there are no more items
    // than CTAs; 2 steps of set-up and epilogue an item, 1 more for its partial, 4 for the
    // merge. Lane c weighs candidate c; the least time wins, then the fewest parts.
    const long long W2 = (long long)red[17] * p.e.r.H_kv, S = p.sms;
    long long cost = 0x7FFFFFFFFFFFFFFFll;
    if (lane < 16 && lane < top) {
      const long long X = (top + lane) / (lane + 1);
      const long long n = (long long)red[lane] * p.e.r.H_kv;
      if (lane == 0 || n <= p.max_split_items) {
        const int waves = ((int)n + p.sms - 1) / p.sms;
        cost = (n <= S ? X * 2 * S : max(X * 2 * S, W2 + X * S)) + (long long)waves * (lane > 0 ? 6 : 4) * S +
               (lane > 0 ? 8 * S : 0);
        cost = cost * 16 + lane;
      }
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) cost = min(cost, __shfl_xor_sync(0xffffffffu, cost, off));
    best = (int)(__shfl_sync(0xffffffffu, cost, 0) & 15);
  }
  const int X = given > 0 ? given : (top + best) / (best + 1);
  pl.longest = X < top ? X : 0;
  // parts, and the prefix of items
  __syncthreads();
  int before = 0;
  for (int b0 = 0; b0 < B; b0 += NT) {
    const int b = b0 + tid;
    int mine = 0;
    if (b < B && pl.blocks[b] > 0) {
      const int s = (pl.parts[b] + X - 1) / X;   // 1 where nothing is cut: X is the longest
      pl.parts[b] = s;
      mine = pl.blocks[b] * s * p.e.r.H_kv;
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += up;
    }
    if (lane == 31) red[warp] = (unsigned long long)incl;
    __syncthreads();
    int base = before, all = 0;
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) base += (int)red[w];
      all += (int)red[w];
    }
    if (b < B) pl.prefix[b] = base + incl - mine;
    before += all;
    __syncthreads();
  }
  if (tid == 0) pl.prefix[B] = before;
  pl.items = before;
  __syncthreads();
  return pl;
}

// One item: a part of the key tiles of one unit.
struct TileItem {
  int id;            // its number; -1: there are no more
  int b, hk, parts;
  SeqTokens s;
  int tok0;          // the unit's first token (of the sequence)
  KeyTiles kt;       // the unit's key tiles ...
  int lo;            // ... of which this part takes list entries lo .. lo + max(n0, n1) - 1
  int n0, n1;        // entries that query tile A / B needs
};
static_assert(sizeof(TileItem) <= 64, "an item slot");

// A sequence's items: groups of `hg` KV heads (their K and V within 64 MiB, half of L2),
// in a group the parts of the key range in turn, in a part the blocks with the last
// (longest) first, the group's heads side by side. (Two, four or more blocks of a head
// side by side, which read the same tiles at the same time, measured no faster: causal,
// 32/8 heads, N = 8192, 402 us with one or two, 412-427 with four to sixteen.)
__device__ __forceinline__ int head_group(const TileParams& p, int len) {
  const long long bytes = (long long)max(len, 1) * p.kv_bytes;
  return (int)max(min((64ll << 20) / bytes, (long long)p.e.r.H_kv), 1ll);
}
__device__ __forceinline__ int tile_item_id(const TilePlan& pl, int b, int hk, int rank, int part, int hg, int H_kv) {
  const int g = hk / hg, gh = min(hg, H_kv - g * hg);
  return pl.prefix[b] + pl.blocks[b] * (pl.parts[b] * g * hg + part * gh) + rank * gh + (hk - g * hg);
}
__device__ __forceinline__ TileItem tile_item_of(const TileParams& p, int id, int b, int hk, int blk, int part, int parts,
                                                 const SeqTokens& s) {
  TileItem it;
  it.id = id;
  it.b = b;
  it.hk = hk;
  it.parts = parts;
  it.s = s;
  it.tok0 = blk * 2 * p.TQ;
  const int first = s.p0 + it.tok0, end = s.p0 + min(it.tok0 + 2 * p.TQ, s.n);
  it.kt = key_tiles_of(first, end, p.e.window, p.e.sinks, p.key_tiles);
  const int all = it.kt.count();
  it.lo = (int)((long long)all * part / parts);
  const int stop = (int)((long long)all * (part + 1) / parts);
  // tile A's last token sees fewer keys than the unit's
  const int endA = s.p0 + min(it.tok0 + p.TQ, s.n);
  const int hiA = min((max(endA, 0) + kPage - 1) / kPage, it.kt.hi);
  const int allA = it.kt.n_sink + max(hiA - it.kt.lo, 0);
  it.n0 = max(min(stop, allA) - it.lo, 0);
  it.n1 = it.tok0 + p.TQ < s.n ? stop - it.lo : 0;
  return it;
}
__device__ __forceinline__ TileItem tile_item(const TileParams& p, const TilePlan& pl, int id) {
  int lo = 0, hi = p.e.r.B;   // prefix[lo] <= id < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.prefix[mid] <= id) lo = mid;
    else hi = mid;
  }
  const SeqTokens s = tile_seq(p, lo);
  const int nb = pl.blocks[lo], parts = pl.parts[lo], hg = head_group(p, s.len);
  int w = id - pl.prefix[lo];
  const int g = w / (nb * parts * hg), gh = min(hg, p.e.r.H_kv - g * hg);
  w -= g * nb * parts * hg;
  const int part = w / (nb * gh);
  w -= part * nb * gh;
  const int rank = w / gh;
  return tile_item_of(p, id, lo, g * hg + (w - rank * gh), nb - 1 - rank, part, parts, s);
}

// Asks for a CTA of this grid that has not been launched: if there is one it will not be,
// and this CTA does its work. The answer (16 bytes) arrives on an mbarrier.
__device__ __forceinline__ void request_cta(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
// The answer: the taken CTA's number, or -1 when none was left.
__device__ __forceinline__ int requested_cta(uint32_t answer) {
  uint32_t some, x;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(some), "=r"(x)
      : "r"(answer)
      : "memory");
  return some ? (int)x : -1;
}

// 16 E4M3 codes of a row to 16-bit values times the row's power of two (a byte; 255:
// a NaN row). Sign-extended to 16 bits and shifted, a code is the 16-bit number with
// its fields in place but the exponent bias off: code * 2^-120 in BF16, code * 2^-8 in
// FP16, subnormal codes included. One multiply by 2^(120 + e) or 2^(8 + e) puts that and the
// row's factor right, exactly: four instructions for two codes, and no conversion (those
// go through the pipe that the softmax's exponentials need).
template <Elem E>
__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (E == Elem::F16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Bytes whose factor is a normal number of the type (the others take widen_slow).
template <Elem E>
__device__ __forceinline__ bool plain_factor(uint32_t byte) {
  return E == Elem::F16 ? byte >= 105 && byte <= 134 : byte <= 134;
}
template <Elem E>
__device__ __forceinline__ void widen16_codes(const uint4& w4, uint32_t f, uint32_t* o) {
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t x;   // two sign-extended codes
    if (k & 1) asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(x) : "r"(w[k >> 1]));
    else asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(x) : "r"(w[k >> 1]));
    o[k] = mul_pair<E>((x << (E == Elem::F16 ? 7 : 4)) & (E == Elem::F16 ? 0xBF80BF80u : 0x87F087F0u), f);
  }
}
// The factor as a pair: the exponent field is byte - 104 (FP16) or byte + 120 (BF16).
template <Elem E>
__device__ __forceinline__ uint32_t factor_pair(uint32_t byte) {
  return E == Elem::F16 ? byte * 0x04000400u - 104u * 0x04000400u : byte * 0x00800080u + 120u * 0x00800080u;
}
// The same for any byte: in two factors where one would leave the type's range.
template <Elem E>
__device__ __noinline__ void widen_slow(uint4 w, uint32_t byte, uint32_t* o) {
  constexpr bool kHalf = E == Elem::F16;
  const float low = exp2f((float)byte - 119.f);
  widen16_codes<E>(w, plain_factor<E>(byte) ? factor_pair<E>(byte)
                      : byte < 134 ? pack_f16x2(low, low) : (kHalf ? 0x78007800u : 0x7F007F00u), o);   // 2^15, 2^127
  if (byte > 134) {
    const float g = exp_factor(byte == 255 ? 255u : byte - 134 + 127);
    const uint32_t f2 = kHalf ? pack_f16x2(g, g) : pack_bf16x2(g, g);
    for (int k = 0; k < 8; ++k) o[k] = mul_pair<E>(o[k], f2);
  }
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

template <int D, Elem E, bool FP8, bool WIN>
__global__ void __launch_bounds__(TCfg<D, FP8>::kThreadsT, 1)
    fa_extend_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const TileParams p) {
  using C = TCfg<D, FP8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::kOffBar + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  __shared__ unsigned long long red[20];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* status = p.e.status;
  const bool paged = p.e.r.table != nullptr;

  if (warp == kWarpProducer && lane == 0) {
    mbar_init(bar(C::kBarQ), 1);
    mbar_init(bar(C::kBarQFree), 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar(C::kBarFull + s), FP8 ? 128 : 1);
      mbar_init(bar(C::kBarEmpty + s), 1);
    }
    for (int X = 0; X < 2; ++X) {
      mbar_init(bar(C::kBarS + X), 1);
      mbar_init(bar(C::kBarP1 + X), 128);
      mbar_init(bar(C::kBarP2 + X), 128);
      mbar_init(bar(C::kBarO + X), 1);
    }
    mbar_init(bar(C::kBarDrain), 1);
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(bar(C::kBarRawFull + s), 1);
      mbar_init(bar(C::kBarRawEmpty + s), 128);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::kBarItem + s), 1);
      mbar_init(bar(C::kBarItemFree + s), C::kItemReaders);
    }
    mbar_init(bar(C::kBarNext), 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // rows TQ * G .. 127 of a tile belong to no token: zero queries, for good (the Q loads
  // write TQ * G rows), so their scores stay finite
  {
    const int used = p.TQ * p.e.G;
    constexpr int kCh = D / 8;   // 16-byte chunks per row; the swizzle permutes within a row
    for (int i = threadIdx.x; i < 2 * (128 - used) * kCh; i += C::kThreadsT) {
      const int X = i / ((128 - used) * kCh), j = i - X * (128 - used) * kCh;
      const int row = used + j / kCh, ch = j % kCh;
      st_shared_v4(sb + C::kOffQ + X * C::kTileBytes + (ch >> 3) * C::kBoxBytes + row * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  // the lengths (and everything else) may come from the previous kernel on the stream
  const TilePlan pl = tile_plan<C::kThreadsT>(p, reinterpret_cast<int*>(smem + C::kOffPlan), red);
  if (p.max_split_items > 0 && threadIdx.x == 0) *p.cut = pl.longest;   // (every CTA that runs: the same value)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  TileItem* slots = reinterpret_cast<TileItem*>(smem + C::kOffItem);
  static_assert(64 % alignof(TileItem) == 0, "item slots are 64 bytes apart");
  auto slot = [&](int q) { return reinterpret_cast<const TileItem*>(reinterpret_cast<uint8_t*>(slots) + 64 * (q & 1)); };
  // item number q (of this CTA) has been published / this warp is done with it
  auto item_ready = [&](int q) { return mbar_wait_w(bar(C::kBarItem + (q & 1)), (uint32_t)(q >> 1) & 1u, s_abort, status); };
  auto item_done = [&](int q) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kBarItemFree + (q & 1)));
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    if (warp == kWarpProducer) {
      // ======================= TMA producer =======================
      if (lane == 0) {
        constexpr int kRing = FP8 ? C::kRaw : C::kStages;
        constexpr int kFullB = FP8 ? C::kBarRawFull : C::kBarFull, kEmptyB = FP8 ? C::kBarRawEmpty : C::kBarEmpty;
        const uint32_t q_bytes = (uint32_t)(2 * p.TQ * p.e.G * D * 2);
        const uint64_t pol = policy_evict_last();
        int tiles = 0, items = 0;   // K/V tile loads issued; items with work
        int asked = 0;              // requests for another CTA
        bool ok = true;
        auto ask = [&]() {
          fence_proxy_async_smem();   // the last answer has been read
          mbar_arrive_expect_tx(bar(C::kBarNext), 16);
          request_cta(sb + C::kOffNext, bar(C::kBarNext));
          ++asked;
        };
        auto next_id = [&]() {
          for (;;) {
            if (!mbar_wait(bar(C::kBarNext), (uint32_t)(asked - 1) & 1u, s_abort, status)) {
              ok = false;
              return -1;
            }
            const int got = requested_cta(sb + C::kOffNext);
            if (got < pl.items) return got;   // an item, or none left
            ask();                            // a CTA past the last item: the grid is an upper bound
          }
        };
        int id = blockIdx.x;
        if (id >= pl.items) {   // (this CTA is one of those: clear away the others)
          ask();
          id = next_id();
        }
        for (int q = 0; ok; ++q) {
          TileItem it;
          it.id = -1;
          if (id >= 0) it = tile_item(p, pl, id);
          if (!mbar_wait(bar(C::kBarItemFree + (q & 1)), ((uint32_t)(q >> 1) & 1u) ^ 1u, s_abort, status)) break;
          *const_cast<TileItem*>(slot(q)) = it;
          mbar_arrive(bar(C::kBarItem + (q & 1)));
          if (id < 0) break;
          ask();   // for the next item, while this one's tiles are loaded
          const int n = max_i(it.n0, it.n1);
          if (n == 0) {
            id = next_id();
            continue;
          }
          if (!mbar_wait(bar(C::kBarQFree), ((uint32_t)items & 1u) ^ 1u, s_abort, status)) {
            ok = false;
            break;
          }
          ++items;
          mbar_arrive_expect_tx(bar(C::kBarQ), q_bytes);
#pragma unroll
          for (int X = 0; X < 2; ++X)
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_5d(sb + C::kOffQ + X * C::kTileBytes + bx * C::kBoxBytes, &tmQ, bar(C::kBarQ), bx * 64, 0,
                          it.s.t0 + it.tok0 + X * p.TQ, it.hk, paged ? 0 : it.b);
          for (int j = 0; j < n && ok; ++j) {
            const int kt = it.kt.tile(it.lo + j);
            int row = 0, slab;
            if (paged) {   // (a page outside the cache: a slab past the end reads as zeros)
              const int pg = page_at(p.e.r, it.b, kt);
              slab = pg >= 0 ? pg * p.e.r.H_kv + it.hk : p.e.r.num_pages * p.e.r.H_kv;
            } else {
              row = kt * 128;
              slab = it.b * p.e.r.H_kv + it.hk;
            }
#pragma unroll
            for (int sel = 0; sel < 2; ++sel, ++tiles) {
              const int st = tiles % kRing;
              if (!mbar_wait(bar(kEmptyB + st), ((uint32_t)(tiles / kRing) & 1u) ^ 1u, s_abort, status)) {
                ok = false;
                break;
              }
              const void* tm = sel ? (const void*)&tmV : (const void*)&tmK;
              if constexpr (FP8) {
                const uint32_t de = sb + C::kOffExp + st * 128;
                const bool real = slab < p.e.r.num_pages * p.e.r.H_kv;
                if (!real) {   // any factor will do for zeros
                  for (int i = 0; i < 128; i += 16) st_shared_v4(de + i, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                  fence_proxy_async_smem();
                }
                mbar_arrive_expect_tx(bar(kFullB + st), C::kRawBytes + (real ? 128 : 0));
                if (real) bulk_copy_1d(de, (sel ? p.e.v_exp : p.e.k_exp) + (size_t)slab * kPage, 128, bar(kFullB + st));
                tma_load_3d_hint(sb + C::kOffRaw + st * C::kRawBytes, tm, bar(kFullB + st), 0, row, slab, pol);
              } else {
                mbar_arrive_expect_tx(bar(kFullB + st), C::kTileBytes);
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  tma_load_3d_hint(sb + C::kOffKV + st * C::kTileBytes + bx * C::kBoxBytes, tm, bar(kFullB + st), bx * 64,
                                   row, slab, pol);
              }
            }
          }
          if (ok) id = next_id();
        }
        // drain: every load issued has landed before the CTA may exit
        if (asked > 0) drain_wait(bar(C::kBarNext), (uint32_t)(asked - 1) & 1u, status);
        if (items > 0) drain_wait(bar(C::kBarQ), (uint32_t)(items - 1) & 1u, status);
        for (int st = 0; st < kRing; ++st) {
          const int k = tiles > st ? (tiles - st + kRing - 1) / kRing : 0;
          if (k > 0) drain_wait(bar(kFullB + st), (uint32_t)(k - 1) & 1u, status);
        }
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ======================= tcgen05 MMA issuer (warp converged) =======================
      constexpr uint32_t idS = idesc_f32(128, 128, false, E);
      constexpr uint32_t idO = idesc_f32(128, D, true, E);
      constexpr uint32_t kStageStep = (uint32_t)(C::kTileBytes >> 4);
      constexpr uint32_t kBox16 = C::kBoxBytes >> 4;
      constexpr uint32_t kHi = desc_sw128_hi(1024);
      const uint32_t lq0 = desc_sw128_lo(sb + C::kOffQ, 16);
      const uint32_t lk0 = desc_sw128_lo(sb + C::kOffKV, 16);
      const uint32_t lv0 = desc_sw128_lo(sb + C::kOffKV, C::kBoxBytes);
      auto issue_S = [&](int X, int st) {
        const uint32_t a0 = lq0 + (uint32_t)X * kStageStep, b0 = lk0 + (uint32_t)st * kStageStep;
        const uint32_t d = tmem + C::tm_s(X);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (uint32_t)(kk >> 2) * kBox16 + (uint32_t)(kk & 3) * 2u;
          mma_ss_lh_w(d, a0 + off, kHi, b0 + off, kHi, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit_w(bar(C::kBarS + X));
      };
      auto issue_PV = [&](int X, int st, bool acc, int h) {   // keys 64 h .. 64 h + 63
        const uint32_t b0 = lv0 + (uint32_t)st * kStageStep;
        const uint32_t d = tmem + C::tm_o(X), a = tmem + C::tm_s(X);
#pragma unroll
        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
          mma_ts_lh_w(d, a + (uint32_t)kk * 8u, b0 + (uint32_t)kk * (16u * 128u >> 4), kHi, idO, (acc || kk > 0) ? 1u : 0u);
      };
      int tiles = 0, items = 0;
      int c0 = 0, c1 = 0;   // tiles of A and B so far: phases of their P barriers
      bool ok = true;
      auto full = [&](int t) {
        ok = mbar_wait_w(bar(C::kBarFull + t % C::kStages), (uint32_t)(t / C::kStages) & 1u, s_abort, status);
        tc_fence_after();
        return ok;
      };
      for (int q = 0; ok; ++q) {
        if (!(ok = item_ready(q))) break;
        const TileItem it = *slot(q);
        item_done(q);
        if (it.id < 0) break;
        const int n = max_i(it.n0, it.n1);
        if (n == 0) continue;
        if (!(ok = mbar_wait_w(bar(C::kBarQ), (uint32_t)items & 1u, s_abort, status))) break;
        ++items;
        if (!full(tiles)) break;
        {
          const int st = tiles % C::kStages;
          if (it.n0 > 0) issue_S(0, st);
          if (it.n1 > 0) issue_S(1, st);
          mma_commit_w(bar(C::kBarEmpty + st));
          if (n == 1) mma_commit_w(bar(C::kBarQFree));
        }
        for (int j = 0; j < n && ok; ++j) {
          const int tV = tiles + 2 * j + 1, tK = tV + 1;
          const int stV = tV % C::kStages, stK = tK % C::kStages;
          const bool next = j + 1 < n;
          if (!full(tV)) break;
          if constexpr (!FP8) {
            // V rows past the sequence's end may hold anything, NaN included, and 0 * NaN
            // is NaN: zero them (contiguous V: the loads filled them with zeros)
            const int key0 = it.kt.tile(it.lo + j) * kPage;
            if (paged && key0 + kPage > it.s.len) {
              const uint32_t base = sb + C::kOffKV + stV * C::kTileBytes;
              const int from = max(it.s.len - key0, 0);
              for (int i = lane; i < (kPage - from) * 8; i += 32)
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  st_shared_v4(base + bx * C::kBoxBytes + (from + (i >> 3)) * 128 + (i & 7) * 16, 0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (j < it.n0) {
            if (!(ok = mbar_wait_w(bar(C::kBarP1 + 0), (uint32_t)c0 & 1u, s_abort, status))) break;
            tc_fence_after();
            issue_PV(0, stV, j > 0, 0);
            if (!(ok = mbar_wait_w(bar(C::kBarP2 + 0), (uint32_t)c0 & 1u, s_abort, status))) break;
            tc_fence_after();
            issue_PV(0, stV, true, 1);
            ++c0;
          }
          if (next) {
            if (!full(tK)) break;
            if (j + 1 < it.n0) issue_S(0, stK);
          }
          if (j < it.n1) {
            if (!(ok = mbar_wait_w(bar(C::kBarP1 + 1), (uint32_t)c1 & 1u, s_abort, status))) break;
            tc_fence_after();
            issue_PV(1, stV, j > 0, 0);
            if (!(ok = mbar_wait_w(bar(C::kBarP2 + 1), (uint32_t)c1 & 1u, s_abort, status))) break;
            tc_fence_after();
            issue_PV(1, stV, true, 1);
            ++c1;
          }
          mma_commit_w(bar(C::kBarEmpty + stV));
          if (next) {
            if (j + 1 < it.n1) issue_S(1, stK);
            mma_commit_w(bar(C::kBarEmpty + stK));
            if (j + 2 == n) mma_commit_w(bar(C::kBarQFree));   // the item's last S
          }
        }
        tiles += 2 * n;
        // each tile's own barrier, so that it never runs ahead of a warpgroup that skips items
        if (it.n0 > 0) mma_commit_w(bar(C::kBarO + 0));
        if (it.n1 > 0) mma_commit_w(bar(C::kBarO + 1));
      }
      // all MMAs done before tensor memory is released
      mma_commit_w(bar(C::kBarDrain));
      drain_wait(bar(C::kBarDrain), 0, status);
      __syncwarp();
    } else if constexpr (FP8) {
      if (warp >= 12) {
        // ======================= code tiles to 16-bit tiles (warps 12-15) =======================
        const int th = threadIdx.x & 127;
        int tiles = 0;
        bool ok = true;
        for (int q = 0; ok; ++q) {
          if (!(ok = item_ready(q))) break;
          const TileItem it = *slot(q);
          item_done(q);
          if (it.id < 0) break;
          const int n = max_i(it.n0, it.n1);
          for (int j = 0; j < 2 * n && ok; ++j, ++tiles) {
            const int rs = tiles % C::kRaw, st = tiles % C::kStages;
            if (!(ok = mbar_wait_w(bar(C::kBarRawFull + rs), (uint32_t)(tiles / C::kRaw) & 1u, s_abort, status))) break;
            if (!(ok = mbar_wait_w(bar(C::kBarEmpty + st), ((uint32_t)(tiles / C::kStages) & 1u) ^ 1u, s_abort, status))) break;
            const uint32_t src = sb + C::kOffRaw + rs * C::kRawBytes;
            const uint32_t dst = sb + C::kOffKV + st * C::kTileBytes;
            const uint32_t exps = sb + C::kOffExp + rs * 128;
            constexpr int kCh = D / 16;        // 16-code chunks per row
            constexpr int kStep = 128 / kCh;   // rows between a thread's chunks: 16 or 32
            // a thread keeps its chunk of the row and its place in the swizzles. At D = 128
            // 16-bit chunks 2 ch of the two boxes share banks: threads of the upper half of
            // the row take the row next door, whose swizzle is odd where theirs is even
            const int ch = th % kCh, row0 = (th / kCh) ^ (ch >> 2);
            const uint32_t from = src + row0 * D + (D == 128 ? ch ^ (row0 & 7) : ch ^ ((row0 >> 1) & 3)) * 16;
            const uint32_t to = dst + (uint32_t)(ch >> 2) * C::kBoxBytes + row0 * 128;
            const uint32_t x0 = (uint32_t)((((2 * ch) & 7) ^ (row0 & 7)) << 4), x1 = x0 ^ 16u;
#pragma unroll 1
            for (int m = 0; m < 128 / kStep; m += 4) {   // four rows in flight
              uint4 w[4];
              uint32_t eb[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                w[i] = ld_shared_v4u(from + (uint32_t)(m + i) * (kStep * D));
                eb[i] = ld_shared_u8(exps + row0 + (uint32_t)(m + i) * kStep);
              }
              const bool plain = plain_factor<E>(eb[0]) && plain_factor<E>(eb[1]) && plain_factor<E>(eb[2]) && plain_factor<E>(eb[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t o[8];
                if (plain) widen16_codes<E>(w[i], factor_pair<E>(eb[i]), o);
                else widen_slow<E>(w[i], eb[i], o);
                const uint32_t at = to + (uint32_t)(m + i) * (kStep * 128);
                st_shared_v4(at + x0, o[0], o[1], o[2], o[3]);
                st_shared_v4(at + x1, o[4], o[5], o[6], o[7]);
              }
            }
            // rows past the sequence's end become zeros
            const int live = paged ? max(it.s.len - it.kt.tile(it.lo + (j >> 1)) * kPage, 0) : kPage;
            if (live < kPage) {
              for (int m = 0; m < 128 / kStep; ++m)
                if (row0 + m * kStep >= live) {   // (this thread's own chunks)
                  const uint32_t at = to + (uint32_t)m * (kStep * 128);
                  st_shared_v4(at + x0, 0u, 0u, 0u, 0u);
                  st_shared_v4(at + x1, 0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(C::kBarFull + st));
            mbar_arrive(bar(C::kBarRawEmpty + rs));
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
    // ======================= softmax warpgroups =======================
    const int X = warp >> 2;
    const int r = (warp & 3) * 32 + lane;   // row within the query tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::tm_s(X), tO = tmem + lane_base + C::tm_o(X);
    const float c = p.e.c;
    const int tr = r / p.e.G, hr = r - tr * p.e.G;   // token of the tile and query head of the group
    const bool in_tile = tr < p.TQ;
    int cnt = 0, items = 0;   // tiles and items of this warpgroup so far: barrier phases
    bool ok = true;
    for (int q = 0; ok; ++q) {
      if (!(ok = item_ready(q))) break;
      // (re-read from shared memory where it is needed: the loop's registers are scarce)
      const volatile TileItem& it = *slot(q);
      if (it.id < 0) break;
      const int n = X ? it.n1 : it.n0;
      const int k_first = it.lo, k_sink = WIN ? it.kt.n_sink : 0, k_skip = WIN ? it.kt.lo - it.kt.n_sink : 0;
      // positions: this row's, and the tile's first and last
      const int pos_lo = it.s.p0 + it.tok0 + X * p.TQ;
      const int pos_hi = pos_lo + p.TQ - 1;
      int pos = min_i(pos_lo + tr, it.s.len - 1);
      // tokens past the block table see no key: then every tile has a mask
      const bool past = (min_i(pos_hi, it.s.p0 + it.s.n - 1) / kPage) >= p.key_tiles;
      if (past && pos / kPage >= p.key_tiles) pos = -1;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++cnt) {
        if (!(ok = mbar_wait(bar(C::kBarS + X), (uint32_t)cnt & 1u, s_abort, status))) break;
        tc_fence_after();
        float s[128];
        tmem_ld32(tS + 0, s);
        tmem_ld32(tS + 32, s + 32);
        tmem_ld32(tS + 64, s + 64);
        tmem_ld32(tS + 96, s + 96);
        tmem_wait_ld();
        const int key0 = (k_first + j + (k_first + j < k_sink ? 0 : k_skip)) * kPage;
        // the mask: keys after a row's position, and those before its window that are no sinks
        const bool cut_hi = past || key0 + kPage - 1 > pos_lo;
        const bool cut_lo = WIN && key0 <= pos_hi - p.e.window && key0 + kPage > p.e.sinks;
        if (cut_hi) {
          const int hi = pos + 1 - key0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= hi) s[i] = -INFINITY;
        }
        if (cut_lo) {
          const int lo = pos + 1 - p.e.window - key0, snk = p.e.sinks - key0;
          if (snk <= 0) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i < lo) s[i] = -INFINITY;
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i < lo && i >= snk) s[i] = -INFINITY;
          }
        }
        // (the scheme of fa_fwd_kernel: exponentials against a reference max that lags by
        // at most 2^tau, decided before P is handed over)
        const bool spec = !__any_sync(0xffffffffu, m_ref == -INFINITY);
        if (!spec) {
          const float m_tile = max_scores<128>(s) * c;
          const bool need = m_tile > m_ref + TileLag<E>::kTau;
          if (__any_sync(0xffffffffu, need)) {
            float alpha = 1.f;
            if (need) {
              alpha = ex2_approx(m_ref - m_tile);   // 0 when there was no reference yet
              m_ref = m_tile;
              l *= alpha;
            }
            if (j > 0) rescale_o<D>(tO, alpha);
          }
        }
        float r1;
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          r1 = exp_half<E>(s, c, m_ref == -INFINITY ? 0.f : m_ref, tS);
          if (!spec || pass > 0) break;
          const float m2 = max_scores<64>(s + 64) * c;
          const bool need = !(r1 <= TileLag<E>::kSumCap) || m2 > m_ref + TileLag<E>::kTau;
          if (!__any_sync(0xffffffffu, need)) break;
          float alpha = 1.f;
          if (need) {
            const float m_new = fmaxf(m_ref, fmaxf(max_scores<64>(s) * c, m2));
            alpha = ex2_approx(m_ref - m_new);
            m_ref = m_new;
            l *= alpha;
          }
          if (j > 0) rescale_o<D>(tO, alpha);
        }
        publish(bar(C::kBarP1 + X));
        const float r2 = exp_half<E>(s + 64, c, m_ref == -INFINITY ? 0.f : m_ref, tS + 32u);
        publish(bar(C::kBarP2 + X));
        l += r1 + r2;
      }
      if (!ok) break;
      if (n > 0) {
        if (!(ok = mbar_wait(bar(C::kBarO + X), (uint32_t)items & 1u, s_abort, status))) break;
        ++items;
        tc_fence_after();
      }
      const int tok = it.tok0 + X * p.TQ + tr;
      const bool live = in_tile && tok < it.s.n;
      // a row that saw no key: O = 0 whatever the products left
      const bool none = !(l > 0.f) && !(l != l);
      if (it.parts == 1) {
        // ---- O / l through the warp's staging rows: a lane holds a row, a store takes kCh
        // lanes a row, so that whole sectors are written (a row's 16 bytes per lane cost
        // 2 us an item: 32 lines a store)
        constexpr int kCh = C::kStgCols / 8, kRows = 32 / kCh;   // 16-byte chunks a row, rows a store
        const float inv = 1.f / l;
        const long long off = it.b * p.o_b + (it.s.t0 + tok) * p.o_t + it.hk * p.o_h + hr * p.o_g;
        const uint32_t stg = sb + C::kOffStg + warp * C::kStgBytes;
        // chunk c of row y lies at y * kCh + (c ^ (y / (8 / kCh)) % kCh): conflict-free both ways
        auto staged = [&](int y, int ch) { return stg + (uint32_t)(y * kCh + (ch ^ ((y / (8 / kCh)) & (kCh - 1)))) * 16u; };
        const unsigned rows = __ballot_sync(0xffffffffu, live);
#pragma unroll 1
        for (int cc = 0; cc < D; cc += C::kStgCols) {
          float ov[C::kStgCols];
          if (n > 0) {
            if constexpr (C::kStgCols == 32) tmem_ld32(tO + cc, ov);
            else tmem_ld16(tO + cc, ov);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < C::kStgCols; ++i) ov[i] = none || n == 0 ? 0.f : ov[i] * inv;
#pragma unroll
          for (int g = 0; g < kCh; ++g)
            st_shared_v4(staged(lane, g), pack2<E>(ov[8 * g], ov[8 * g + 1]), pack2<E>(ov[8 * g + 2], ov[8 * g + 3]),
                         pack2<E>(ov[8 * g + 4], ov[8 * g + 5]), pack2<E>(ov[8 * g + 6], ov[8 * g + 7]));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kCh; ++i) {
            const int y = i * kRows + lane / kCh, ch = lane % kCh;
            const long long at = __shfl_sync(0xffffffffu, off, y);
            const float4 v = ld_shared_v4f(staged(y, ch));
            if (rows >> y & 1)
              st_global_v4(static_cast<uint16_t*>(p.e.o) + at + cc + 8 * ch, __float_as_uint(v.x), __float_as_uint(v.y),
                           __float_as_uint(v.z), __float_as_uint(v.w));
          }
          __syncwarp();
        }
        if (live && p.e.lse) p.e.lse[off / D] = none ? -INFINITY : (m_ref + __log2f(l)) * kLn2;
      } else {
        // ---- partial: [16-byte chunk][row], so a warp's rows are contiguous
        const int row = X * 128 + r;
        const int item = it.id;
        float4* po = reinterpret_cast<float4*>(p.e.part_o) + (size_t)item * (D / 4) * kBlockRows + row;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float ov[32];
          if (n > 0) {
            tmem_ld32(tO + cc, ov);
            tmem_wait_ld();
          }
          if (n > 0 && live && FA_DBG_OK(status, item < p.max_split_items)) {
#pragma unroll
            for (int g = 0; g < 8; ++g)
              __stcg(po + (size_t)(cc / 4 + g) * kBlockRows,
                     none ? make_float4(0.f, 0.f, 0.f, 0.f)
                          : make_float4(ov[4 * g], ov[4 * g + 1], ov[4 * g + 2], ov[4 * g + 3]));
          }
        }
        if (live && FA_DBG_OK(status, item < p.max_split_items))
          __stcg(reinterpret_cast<float2*>(p.e.part_ml) + (size_t)item * kBlockRows + row,
                 make_float2(none ? -INFINITY : m_ref, none ? 0.f : l));
      }
      tc_fence_before();   // O is read before the next item's first P V (ordered by its P)
      item_done(q);
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Combines the parts of each split unit: M = max m, L = sum 2^(m - M) l, O = sum
// 2^(m - M) O / L. Work is one 128-row tile of a unit by 32 columns, one thread a row,
// so that the loads of all parts are in flight and coalesced over rows.
template <int D, Elem E>
__global__ void __launch_bounds__(128) fa_extend_tile_merge_kernel(const TileParams p) {
  __shared__ int mem[kTileMaxSeqs * 3 + 4];
  __shared__ unsigned long long red[20];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cut = __ldcg(p.cut);
  if (cut == 0) return;   // whole units: the main kernel finished them
  const TilePlan pl = tile_plan<128>(p, mem, red, cut);
  constexpr int kCols = 32, kPer = 2 * (D / kCols);
  const int r = threadIdx.x;
  const int tr = r / p.e.G, hr = r - tr * p.e.G;
  for (int w = blockIdx.x;; w += gridDim.x) {
    int item = w / kPer;
    const int sub = w - item * kPer, X = sub & 1, c0 = (sub >> 1) * kCols;
    // the item-th unit of the split sequences, as the item of its part 0
    int b = 0, base = 0;
    for (; b < p.e.r.B; ++b) {
      const int n = pl.parts[b] > 1 ? pl.blocks[b] * p.e.r.H_kv : 0;
      if (item < base + n) break;
      base += n;
    }
    if (b == p.e.r.B) break;
    const int nb = pl.blocks[b], u = item - base;
    const SeqTokens sq = tile_seq(p, b);
    const int hg = head_group(p, sq.len), hk = u / nb, rank = u - hk * nb;
    item = tile_item_id(pl, b, hk, rank, 0, hg, p.e.r.H_kv);
    const int step = nb * min(hg, p.e.r.H_kv - hk / hg * hg);   // items between parts
    const TileItem it = tile_item_of(p, item, b, hk, nb - 1 - rank, 0, pl.parts[b], sq);
    const int tok = it.tok0 + X * p.TQ + tr;
    if (tr >= p.TQ || tok >= it.s.n) continue;
    const size_t row = (size_t)X * 128 + r;
    const float2* ml = reinterpret_cast<const float2*>(p.e.part_ml);
    float M = -INFINITY, L = 0.f;
    for (int z = 0; z < it.parts; ++z) {
      const float2 v = __ldcg(ml + (size_t)(item + z * step) * kBlockRows + row);
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
    float a[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) a[i] = 0.f;
    for (int z = 0; z < it.parts; ++z) {
      const float2 v = __ldcg(ml + (size_t)(item + z * step) * kBlockRows + row);
      const bool live = v.y > 0.f || v.y != v.y;
      const float m = live ? ex2_approx(v.x - M) : 0.f;
      L += m * v.y;
      if (live) {   // (a part without a visible key wrote no O)
        const float4* src = reinterpret_cast<const float4*>(p.e.part_o) +
                            ((size_t)(item + z * step) * (D / 4) + c0 / 4) * kBlockRows + row;
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) {
          const float4 x = __ldcg(src + (size_t)c * kBlockRows);
          a[4 * c] += m * x.x; a[4 * c + 1] += m * x.y; a[4 * c + 2] += m * x.z; a[4 * c + 3] += m * x.w;
        }
      }
    }
    const float inv = L > 0.f ? 1.f / L : (L != L ? L : 0.f);
    const long long off = it.b * p.o_b + (it.s.t0 + tok) * p.o_t + it.hk * p.o_h + hr * p.o_g;
    uint16_t* dst = static_cast<uint16_t*>(p.e.o) + off + c0;
#pragma unroll
    for (int c = 0; c < kCols; c += 8)
      st_global_v4(dst + c, pack2<E>(a[c] * inv, a[c + 1] * inv), pack2<E>(a[c + 2] * inv, a[c + 3] * inv),
                   pack2<E>(a[c + 4] * inv, a[c + 5] * inv), pack2<E>(a[c + 6] * inv, a[c + 7] * inv));
    if (c0 == 0 && p.e.lse) p.e.lse[off / D] = L > 0.f ? (M + __log2f(L)) * kLn2 : (L != L ? L : -INFINITY);
  }
}

template <int D, Elem E, bool FP8, bool WIN>
cudaError_t launch_tile_t2(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TileParams& p,
                           cudaStream_t stream) {
  using C = TCfg<D, FP8>;
  static bool attr[64] = {false};   // per device; a repeated set is harmless
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!attr[dev]) {
    cudaError_t e = cudaFuncSetAttribute(fa_extend_tile_kernel<D, E, FP8, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  cudaError_t e = launch_kernel(fa_extend_tile_kernel<D, E, FP8, WIN>, dim3((unsigned)p.grid), dim3(C::kThreadsT), C::kSmemBytes,
                                stream, tq, tk, tv, p);
  if (e != cudaSuccess || p.max_split_items == 0) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(8 * p.sms));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_extend_tile_merge_kernel<D, E>, p);
}

}  // namespace

cudaError_t launch_tile(int d, int dtype, int format, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const TileParams& p, cudaStream_t stream) {
  const bool fp8 = format == FA_CACHE_E4M3, win = p.e.window > 0;
#define FA_TILE_GO(DD, EE)                                                                 \
  return fp8 ? (win ? launch_tile_t2<DD, EE, true, true>(tq, tk, tv, p, stream)           \
                    : launch_tile_t2<DD, EE, true, false>(tq, tk, tv, p, stream))         \
             : (win ? launch_tile_t2<DD, EE, false, true>(tq, tk, tv, p, stream)          \
                    : launch_tile_t2<DD, EE, false, false>(tq, tk, tv, p, stream))
  if (dtype == FA_DTYPE_FP16) {
    if (d == 128) FA_TILE_GO(128, Elem::F16);
    FA_TILE_GO(64, Elem::F16);
  }
  if (d == 128) FA_TILE_GO(128, Elem::BF16);
  FA_TILE_GO(64, Elem::BF16);
#undef FA_TILE_GO
}

}  // namespace fa
