// Exact attention backward for sm_103a: dQ, dK, dV of O = softmax(scale Q K^T) V.
//
// The backward recomputes the scores tile by tile from Q, K and the per-row
// log-sum-exp the forward saved, instead of storing the N x N matrices ("Why
// is standard attention memory-bound...", Step 4; "Why does the backward pass
// recompute the scores?"). With P = exp(S - LSE) rebuilt exactly:
//   dV = P^T dO,  dP = dO V^T,  D = rowsum(dO * O),  dS = P * (dP - D),
//   dQ = scale dS K,  dK = scale dS^T Q.
//
// Two launches on the caller's stream:
//  * fa_bwd_prep_kernel: per query row, lse2 = LSE log2(e) (+inf where the row
//    sees no key, and on the padding rows of the last tile) and D, into arrays
//    padded to whole 128-row tiles.
//  * fa_bwd_kernel, whose CTAs take one of two roles (they share no data, so
//    both run in one grid, the dK/dV CTAs before the dQ CTAs):
//    - dK/dV: one CTA per (batch, KV head, block of 128 keys). K and V of the
//      block stay in shared memory; the CTA walks the query tiles of every
//      query head that reads the KV head (GQA sums them in place, no atomics).
//      Keys are the TMEM lanes: S^T = K Q^T and dP^T = V dO^T (SS MMAs), then
//      each thread (one key) turns its row into P^T and dS^T (BF16 or FP16,
//      written back over its S^T / dP^T columns) and the MMA warp accumulates
//      dV += P^T dO and dK += dS^T Q with A read from tensor memory.
//    - dQ: one CTA per (batch, query head, 128-row tile); query rows are the
//      TMEM lanes: S = Q K^T, dP = dO V^T, then dS, then dQ += dS K.
//    In either role the products of a step are issued as  A(i) S(i+1) B(i) dP(i+1)
//    (bwd_mma), so that the element-wise warps work on S while the tensor core makes B
//    and dP, and on dP while it makes A and S.
// Every operand form is one the forward kernel uses: K-major SW128 tiles for
// the score-shaped products, A from tensor memory with an MN-major B for the
// accumulating ones. S and dP are computed twice (once per role): 14 N^2 d
// FLOPs of work for the 10 N^2 d of the usual count, in exchange for no
// atomic accumulation and deterministic results.
//
// Sliding window with sinks (WIN = true, fa_backward_window): the same two roles over
// fewer tiles. A dK/dV CTA walks the query tiles from the first row that sees its block
// to the last one whose window reaches it; a block that holds sink keys is seen by all
// later rows, so its steps are cut over several CTAs, which go first and leave FP32
// partials (fa_bwd_sink_kernel adds them in order). A dQ CTA walks the sink blocks,
// then its window's. WIN = false compiles to the code without any of it.
// There the roles are two launches, dQ first, because dQ also puts D right. D from the
// 16-bit O is off by O's rounding, D~ = D - r, and where a row's weight sits on one key, dP
// and D cancel and the error shows (a training step with a hundredth of its keys eight times
// larger: dQ and dK 0.8 % off). But the exact dS sum to 0 over a row, so r is the
// row's sum of dS~ = P (dP - D~), kept in FP32; dQ = scale (dS~ K - r (P K)) with one more
// accumulating product, and dK/dV start from D~ + r.
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_serving.cuh"
#include "fa_window.h"

#include <cmath>

namespace fa {
namespace {

// warps 0-7 element-wise: two warpgroups on the same 128 TMEM lanes, warpgroup g
// taking columns [32g, 32g+32) of every 64-column half; warp 8 TMA, warp 9 MMA
constexpr int kBwdThreads = 320;
constexpr int kBwdEwThreads = 256;
constexpr int kBwdWarpProducer = 8;
constexpr int kBwdWarpMma = 9;
constexpr int kT = 128;            // query rows per tile = keys per block
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
  int B, H_q, H_kv, N_q, N_k, G;
  int causal, kv_off;      // kv_off = N_k - N_q: row i sees key j iff j <= i + kv_off
  int n_qt, n_kb, nq_pad;  // query tiles, key blocks, n_qt * 128
  int window, sinks, n_sb; // WIN: the mask, and the key blocks that hold sinks,
  int sink_parts;          // each cut over this many CTAs,
  float* part;             // whose partials (more than one) are [CTA][dV, dK][D / 4][128 keys] float4
  float c;                 // scale * log2(e)
  float scale;
  const float* lse2;       // [B*H_q][nq_pad]
  float* dsum;             // [B*H_q][nq_pad]
  void* dq;                // [B][H_q][N_q][d]
  void* dk;                // [B][H_kv][N_k][d]
  void* dv;
  int* status;
};

// The products of one pass over the streamed tiles (bwd_mma).
enum class Pass : int { kDkDv, kDq, kDqSum };   // kDqSum: dQ with P K beside it

template <int D>
struct BwdCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = 128 * 128;        // 128 rows x 128 bytes
  static constexpr int kTileBytes = kT * D * 2;
  static constexpr int kVecBytes = kT * 4;
  // Two resident tiles, and two rings of streamed ones: X (Q for dK/dV, K for dQ), which
  // the score product of a step reads first and its last accumulating product still
  // needs, half a step before the slot two on is wanted: three slots; and Y (dO or V): two.
  static constexpr int kX = 3, kY = 2;
  static constexpr int kOffRes = 0;
  static constexpr int kOffX = 2 * kTileBytes;
  static constexpr int kOffY = kOffX + kX * kTileBytes;
  // dK/dV: lse2 of each Y slot (read while it is held), D of each X slot; dQ: its rows' own
  static constexpr int kOffLse = kOffY + kY * kTileBytes;
  static constexpr int kOffD = kOffLse + kY * kVecBytes;
  static constexpr int kOffBar = kOffD + kX * kVecBytes;
  // kBarRes + i: resident tile i; kBarS, kBarDp: a step's products done; kBarP: P stored (or,
  // where no product takes it, S read); kBarDs: dS stored
  static constexpr int kBarRes = 0, kBarXFull = 2, kBarXEmpty = kBarXFull + kX, kBarYFull = kBarXEmpty + kX,
                       kBarYEmpty = kBarYFull + kY, kBarS = kBarYEmpty + kY, kBarDp = kBarS + 1, kBarP = kBarS + 2,
                       kBarDs = kBarS + 3, kBarDone = kBarS + 4, kBarDrain = kBarS + 5, kNumBars = kBarS + 6;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16;   // (the array is declared 1024-byte aligned)
  // launched with at least 116 KiB so that one CTA holds an SM: each CTA takes all
  // 512 tensor-memory columns, and a second one would only wait in its allocation
  static constexpr int kLaunchSmem = kSmemBytes < 116 * 1024 ? 116 * 1024 : kSmemBytes;
  static_assert(kLaunchSmem <= 227 * 1024, "shared memory");
  static constexpr uint32_t kTmemCols = 512;
  // tensor memory: [0,128) S or S^T, [128,256) dP or dP^T, each as two chunks of 64
  // columns, one per warpgroup; the 16-bit P / P^T or dS / dS^T of a chunk's 64 keys or
  // rows is packed over the chunk's own first 32 columns (so neither warpgroup
  // writes a column the other still reads); [256,256+D) dV, or P K; [384,384+D) dK or dQ
  static constexpr uint32_t kTmS = 0, kTmP = 128, kTmA = 256, kTmB = 384;
};

// Tensor-memory column of the packed 16-bit operand for K-step kk (16 rows or
// keys): chunk kk / 4, its first 32 columns.
__device__ __forceinline__ uint32_t packed_col(int kk) { return (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u; }

__device__ __forceinline__ void bwd_publish(uint32_t bar) {
  tmem_wait_st();
  tc_fence_before();
  mbar_arrive(bar);
}

__device__ __forceinline__ void bwd_drain_wait(uint32_t bar, uint32_t parity, int* status) {
  volatile int never = 0;
  mbar_wait(bar, parity, &never, status);
}

// A 16-bit element of either type widened to FP32.
template <Elem E>
__device__ __forceinline__ float widen16(uint16_t bits) {
  if constexpr (E == Elem::F16) return __half2float(__ushort_as_half(bits));
  else return __uint_as_float((uint32_t)bits << 16);
}

// One row of 128 x D FP32 tensor-memory columns (this thread's lane) to global
// memory as 16-bit values times `mul`; `zero` writes zeros instead (no MMA ran).
// Called by every lane of the warp with warp-uniform `zero` (the tensor-memory
// load is a warp-collective instruction); only lanes with `valid` store.
// Columns [c0, c1), multiples of 32.
template <int D, Elem E>
__device__ __forceinline__ void store_row(uint32_t t_row, uint16_t* dst, float mul, bool zero, bool valid,
                                          int c0 = 0, int c1 = D) {
#pragma unroll 1
  for (int cc = c0; cc < c1; cc += 32) {
    float v[32];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    } else {
      tmem_ld32(t_row + (uint32_t)cc, v);
      tmem_wait_ld();
    }
    if (!valid) continue;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      st_global_v4(dst + cc + 8 * g, pack2<E>(v[8 * g] * mul, v[8 * g + 1] * mul),
                   pack2<E>(v[8 * g + 2] * mul, v[8 * g + 3] * mul), pack2<E>(v[8 * g + 4] * mul, v[8 * g + 5] * mul),
                   pack2<E>(v[8 * g + 6] * mul, v[8 * g + 7] * mul));
  }
}

// lse2 and D per query row, padded to whole tiles. One warp per four padded rows (of
// one tile, as n_rows is a multiple of 128), their loads in flight together: with one row a
// warp the 134 MB of 32 heads x 8192 rows took 44 us, block launches in the way.
constexpr int kPrepRows = 4;
template <int D, Elem E>
__global__ void __launch_bounds__(256) fa_bwd_prep_kernel(const uint16_t* o, const uint16_t* dout,
                                                          const float* lse, float* lse2, float* dsum,
                                                          int N_q, int nq_pad, long long n_rows) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long w0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kPrepRows;
  if (w0 >= n_rows) return;
  const long long bh = w0 / nq_pad;
  const int r0 = (int)(w0 - bh * nq_pad);
  constexpr int kPer = D / 32;   // elements per lane (2 or 4), one 4- or 8-byte load each
  uint32_t wo[kPrepRows][2], wd[kPrepRows][2];
  float l[kPrepRows];
#pragma unroll
  for (int x = 0; x < kPrepRows; ++x) {
    if (r0 + x >= N_q) continue;
    const size_t row = ((size_t)bh * N_q + r0 + x) * D;
    if constexpr (kPer == 4) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(o + row) + lane);
      const uint2 b = __ldg(reinterpret_cast<const uint2*>(dout + row) + lane);
      wo[x][0] = a.x; wo[x][1] = a.y;
      wd[x][0] = b.x; wd[x][1] = b.y;
    } else {
      wo[x][0] = __ldg(reinterpret_cast<const uint32_t*>(o + row) + lane);
      wd[x][0] = __ldg(reinterpret_cast<const uint32_t*>(dout + row) + lane);
    }
    l[x] = __ldg(lse + (size_t)bh * N_q + r0 + x);
  }
#pragma unroll
  for (int x = 0; x < kPrepRows; ++x) {
    if (r0 + x >= N_q) {
      if (lane == 0) {
        lse2[w0 + x] = INFINITY;
        dsum[w0 + x] = 0.f;
      }
      continue;
    }
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int sh = 16 * (i & 1);
      acc += widen16<E>((uint16_t)(wo[x][i >> 1] >> sh)) * widen16<E>((uint16_t)(wd[x][i >> 1] >> sh));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (lane == 0) {
      lse2[w0 + x] = (l[x] == -INFINITY) ? INFINITY : l[x] * kLog2e;
      dsum[w0 + x] = acc;
    }
  }
}

// What both roles share. Barriers and tensor memory; returns the allocation. The loading
// thread issues its first loads (`first`) as soon as the barriers stand.
template <int D, typename F>
__device__ __forceinline__ uint32_t bwd_setup(uint8_t* smem, int warp, int lane, F first) {
  using C = BwdCfg<D>;
  const uint32_t bars = smem_u32(smem) + C::kOffBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  if (warp == kBwdWarpProducer && lane == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bars + 8 * i, i == C::kBarP || i == C::kBarDs ? kBwdEwThreads : 1);
    *reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4) = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kBwdWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  // the next kernel may set itself up on the SMs that this one's last CTAs leave free, as
  // this one did: nothing in global memory has been touched up to here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == kBwdWarpProducer && lane == 0) first();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *tmem_slot;
}

// One tile of 128 rows from row r0 of slab `slab`.
template <int D>
__device__ __forceinline__ void bwd_load_tile(uint32_t dst, const CUtensorMap& map, uint32_t bar, int r0, int slab) {
  using C = BwdCfg<D>;
#pragma unroll
  for (int bx = 0; bx < C::kBoxes; ++bx) tma_load_3d(dst + bx * C::kBoxBytes, &map, bar, bx * 64, r0, slab);
}

// Every load issued (nx, ny into the rings) has landed before the CTA may exit.
template <int D>
__device__ __forceinline__ void bwd_drain_loads(uint32_t bars, int nx, int ny, int* status) {
  using C = BwdCfg<D>;
  for (int i = 0; i < 2; ++i) bwd_drain_wait(bars + 8 * (C::kBarRes + i), 0, status);
  for (int s = 0; s < C::kX; ++s)
    if (nx > s) bwd_drain_wait(bars + 8 * (C::kBarXFull + s), (uint32_t)((nx - 1 - s) / C::kX) & 1u, status);
  for (int s = 0; s < C::kY; ++s)
    if (ny > s) bwd_drain_wait(bars + 8 * (C::kBarYFull + s), (uint32_t)((ny - 1 - s) / C::kY) & 1u, status);
}

// The MMA warp, n >= 1 steps: with the resident tiles R0, R1 and step i's X, Y,
//   S = R0 X^T,  dP = R1 Y^T                       (K, Q and V, dO; or Q, K and dO, V)
//   A += P Y  (dV; kDqSum: P X, that is P K; kDq: none),   B += dS X  (dK or dQ)
// in the order  A(i) S(i+1) B(i) dP(i+1),  all products 128 x 128: while the tensor core
// makes B(i) and dP(i+1) the element-wise warps turn S(i+1) into P, and dP(i+1) into dS
// while it makes A(i+1) and S(i+2). S(i+1) goes over the columns of P(i), dP(i+1) over dS(i):
// MMAs run in the order of issue. Halves of 64 columns in turn (N = 64, each half's
// products and element-wise pass overlapping the other's) took 786 us for 32 heads x 4096
// rows, this 682 (654 with the CTAs in today's order: 1050 TFLOP/s of the usual count,
// 1470 of what is issued): an MMA
// with N = 64 reads all of A from shared memory for half the work. With P and dS published in
// two halves, each product started on the first: 723 us. What bounds a step now is
// shared memory (S and dP read 128 bytes a cycle of it, and the tiles come in through it) and
// the handoffs: 3000 of its 3400 cycles remain when the element-wise warps compute nothing.
template <int D, Elem E, Pass R>
__device__ __forceinline__ void bwd_mma(uint32_t sb, uint32_t tmem, int n, volatile int* s_abort, int* status) {
  using C = BwdCfg<D>;
  constexpr uint32_t idS = idesc_f32(128, kT, false, E);
  constexpr uint32_t idO = idesc_f32(128, D, true, E);
  constexpr uint32_t kHi = desc_sw128_hi(1024);
  constexpr uint32_t kBox16 = C::kBoxBytes >> 4;
  auto bar = [&](int i) -> uint32_t { return sb + C::kOffBar + 8 * i; };
  auto wait = [&](int i, uint32_t parity) { return mbar_wait_w(bar(i), parity & 1u, s_abort, status); };
  auto tile_x = [&](int i) { return sb + C::kOffX + (i % C::kX) * C::kTileBytes; };
  auto tile_y = [&](int i) { return sb + C::kOffY + (i % C::kY) * C::kTileBytes; };
  // K-steps of 16 over d, both operands K-major
  auto scores = [&](uint32_t col, uint32_t a, uint32_t b, int done) {
    const uint32_t la = desc_sw128_lo(a, 16), lb = desc_sw128_lo(b, 16);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = (uint32_t)(kk >> 2) * kBox16 + (uint32_t)(kk & 3) * 2u;
      mma_ss_lh_w(tmem + col, la + off, kHi, lb + off, kHi, idS, kk > 0 ? 1u : 0u);
    }
    mma_commit_w(bar(done));
  };
  // K-steps of 16 over the tile's rows: A from tensor memory, the row-major tile as an MN-major operand
  auto accumulate = [&](uint32_t acc, uint32_t col, uint32_t tile, bool first) {
    const uint32_t lb = desc_sw128_lo(tile, C::kBoxBytes);
#pragma unroll
    for (int kk = 0; kk < kT / 16; ++kk)
      mma_ts_lh_w(tmem + acc, tmem + col + packed_col(kk), lb + (uint32_t)kk * (16u * 128u >> 4), kHi, idO,
                  !first || kk > 0 ? 1u : 0u);
  };
  auto s_product = [&](int i) {
    if (!wait(C::kBarXFull + i % C::kX, (uint32_t)(i / C::kX))) return false;
    tc_fence_after();
    scores(C::kTmS, sb + C::kOffRes, tile_x(i), C::kBarS);
    return true;
  };
  auto dp_product = [&](int i) {
    if (!wait(C::kBarYFull + i % C::kY, (uint32_t)(i / C::kY))) return false;
    tc_fence_after();
    scores(C::kTmP, sb + C::kOffRes + C::kTileBytes, tile_y(i), C::kBarDp);
    if constexpr (R != Pass::kDkDv) mma_commit_w(bar(C::kBarYEmpty + i % C::kY));   // V's last reader
    return true;
  };
  bool ok = wait(C::kBarRes, 0) && s_product(0) && wait(C::kBarRes + 1, 0) && dp_product(0);
  for (int i = 0; i < n && ok; ++i) {
    if (!(ok = wait(C::kBarP, (uint32_t)i))) break;
    tc_fence_after();
    if constexpr (R == Pass::kDkDv) {
      accumulate(C::kTmA, C::kTmS, tile_y(i), i == 0);
      mma_commit_w(bar(C::kBarYEmpty + i % C::kY));
    } else if constexpr (R == Pass::kDqSum) {
      accumulate(C::kTmA, C::kTmS, tile_x(i), i == 0);
    }
    if (i + 1 < n && !(ok = s_product(i + 1))) break;
    if (!(ok = wait(C::kBarDs, (uint32_t)i))) break;
    tc_fence_after();
    accumulate(C::kTmB, C::kTmP, tile_x(i), i == 0);
    mma_commit_w(bar(C::kBarXEmpty + i % C::kX));
    if (i + 1 < n) ok = dp_product(i + 1);
  }
  mma_commit_w(bar(C::kBarDone));
  mma_commit_w(bar(C::kBarDrain));
  bwd_drain_wait(bar(C::kBarDrain), 0, status);
}

// ---------------------------------------------------------------- dK, dV
template <int D, Elem E, bool WIN>
__device__ __forceinline__ void bwd_dkdv_cta(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                             const CUtensorMap& tmdO, const BwdParams& p, int bhk, int kb,
                                             int part = 0, int parts = 1) {
  using C = BwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::kOffBar + 8 * i; };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int b = bhk / p.H_kv, hk = bhk - b * p.H_kv;
  const int j0 = kb * kT;
  // query tiles that see at least one key of the block
  int t_lo = 0;
  if (p.causal) {
    const int first = j0 - p.kv_off;                // the first row that sees key j0
    t_lo = first <= 0 ? 0 : first / kT;
  }
  int t_hi = p.n_qt;
  if constexpr (WIN) {
    if (j0 >= p.sinks) {   // the last row that sees a key of the block sees its last one
      const int last = min(j0 + kT, p.N_k) - 1 + p.window - 1 - p.kv_off;
      t_hi = last < 0 ? 0 : min(p.n_qt, last / kT + 1);
    }
  }
  const int n_t = t_lo < t_hi ? t_hi - t_lo : 0;
  // WIN: the steps i0 .. i0 + n_steps - 1 of the block's, in a CTA that has a part of them
  const int i0 = WIN ? (int)((long long)p.G * n_t * part / parts) : 0;
  const int n_steps = WIN ? (int)((long long)p.G * n_t * (part + 1) / parts) - i0 : p.G * n_t;

  // step i's tiles: Q with D of its rows, dO with lse2 (FA_DEBUG: false when not in their tensors)
  auto load_x = [&](int i) {
    const int hl = (i0 + i) / n_t, q0 = (t_lo + (i0 + i - hl * n_t)) * kT, x = i % C::kX;
    const int bhq = b * p.H_q + hk * p.G + hl;
    if (!FA_DBG_OK(p.status, q0 + kT <= p.nq_pad && bhq < p.B * p.H_q)) return false;
    mbar_arrive_expect_tx(bar(C::kBarXFull + x), C::kTileBytes + C::kVecBytes);
    bwd_load_tile<D>(sb + C::kOffX + x * C::kTileBytes, tmQ, bar(C::kBarXFull + x), q0, bhq);
    bulk_copy_1d(sb + C::kOffD + x * C::kVecBytes, p.dsum + (size_t)bhq * p.nq_pad + q0, C::kVecBytes,
                 bar(C::kBarXFull + x));
    return true;
  };
  auto load_y = [&](int i) {
    const int hl = (i0 + i) / n_t, q0 = (t_lo + (i0 + i - hl * n_t)) * kT, y = i % C::kY;
    const int bhq = b * p.H_q + hk * p.G + hl;
    mbar_arrive_expect_tx(bar(C::kBarYFull + y), C::kTileBytes + C::kVecBytes);
    bwd_load_tile<D>(sb + C::kOffY + y * C::kTileBytes, tmdO, bar(C::kBarYFull + y), q0, bhq);
    bulk_copy_1d(sb + C::kOffLse + y * C::kVecBytes, p.lse2 + (size_t)bhq * p.nq_pad + q0, C::kVecBytes,
                 bar(C::kBarYFull + y));
  };
  const uint32_t tmem = bwd_setup<D>(smem, warp, lane, [&] {
    if (n_steps == 0) return;
    mbar_arrive_expect_tx(bar(C::kBarRes), C::kTileBytes);
    bwd_load_tile<D>(sb + C::kOffRes, tmK, bar(C::kBarRes), j0, bhk);
    load_x(0);
    mbar_arrive_expect_tx(bar(C::kBarRes + 1), C::kTileBytes);
    bwd_load_tile<D>(sb + C::kOffRes + C::kTileBytes, tmV, bar(C::kBarRes + 1), j0, bhk);
    load_y(0);
  });

  if (warp == kBwdWarpProducer) {
    if (lane == 0 && n_steps > 0) {
      int nx = 1, ny = 1;
      for (int i = 1; i < n_steps; ++i) {
        const int x = i % C::kX, y = i % C::kY;
        if (!mbar_wait(bar(C::kBarXEmpty + x), ((uint32_t)(i / C::kX) & 1u) ^ 1u, s_abort, p.status)) break;
        if (!load_x(i)) break;   // reported, not loaded (the consumer's bounded wait then gives up)
        ++nx;
        if (!mbar_wait(bar(C::kBarYEmpty + y), ((uint32_t)(i / C::kY) & 1u) ^ 1u, s_abort, p.status)) break;
        load_y(i);
        ++ny;
      }
      bwd_drain_loads<D>(sb + C::kOffBar, nx, ny, p.status);
    }
    __syncwarp();
  } else if (warp == kBwdWarpMma) {
    if (n_steps > 0) bwd_mma<D, E, Pass::kDkDv>(sb, tmem, n_steps, s_abort, p.status);
    __syncwarp();
  } else if (warp < 8) {
    // ---- element-wise: this thread is key k of the block (TMEM lane k), in
    // warpgroup grp, which takes the 64-row chunk grp of every tile
    const int grp = warp >> 2;
    const int k = (warp & 3) * 32 + lane;
    const int key = j0 + k;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int r0 = 64 * grp;
    const uint32_t tS = tmem + lane_base + C::kTmS + r0, tP = tmem + lane_base + C::kTmP + r0;
    const float c = p.c;
    bool ok = true;
    for (int i = 0; i < n_steps && ok; ++i) {
      const int x = i % C::kX, y = i % C::kY;
      const int hl = (i0 + i) / n_t, t = t_lo + (i0 + i - hl * n_t);
      // rows with key > row + kv_off are masked (causal): rows below r_min see no key k;
      // WIN: nor do rows from r_max on, whose window has passed it
      const int r_min = p.causal ? key - p.kv_off - t * kT : -1;
      const int r_max = WIN && key >= p.sinks ? r_min + p.window : 0x7FFFFFFF;
      // the vectors came by TMA: observe their barriers directly (neither can move on
      // before this thread publishes what it makes of them)
      if (!(ok = mbar_wait_w(bar(C::kBarS), (uint32_t)i & 1u, s_abort, p.status) &&
                 mbar_wait_w(bar(C::kBarYFull + y), (uint32_t)(i / C::kY) & 1u, s_abort, p.status)))
        break;
      tc_fence_after();
      if (!FA_DBG_OK(p.status, tmem_in(lane_base + C::kTmS + r0, 64) && tmem_in(lane_base + C::kTmP + r0, 64))) {
        ok = false;   // FA_DEBUG: reported; this step is not processed
        break;
      }
      float s[64], dp[64];
      tmem_ld32(tS, s);
      tmem_ld32(tS + 32, s + 32);
      tmem_wait_ld();
      // most tiles lie inside the window (or below the diagonal) of all their rows: the mask
      // is a pass of its own, over scores, where some row of the warp's chunk needs it
      if (__any_sync(0xffffffffu, r0 < r_min || r0 + 64 > r_max)) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (r0 + e < r_min || r0 + e >= r_max) s[e] = -INFINITY;
      }
      uint32_t pk[32];
      const float4* vl = reinterpret_cast<const float4*>(smem + C::kOffLse + y * C::kVecBytes) + r0 / 4;
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        const float4 l = vl[e / 4];
        s[e] = ex2_approx(s[e] * c - l.x);
        s[e + 1] = ex2_approx(s[e + 1] * c - l.y);
        s[e + 2] = ex2_approx(s[e + 2] * c - l.z);
        s[e + 3] = ex2_approx(s[e + 3] * c - l.w);
        pk[e / 2] = pack2<E>(s[e], s[e + 1]);
        pk[e / 2 + 1] = pack2<E>(s[e + 2], s[e + 3]);
      }
      // P^T of the chunk's 64 rows over its own first 32 columns (read above)
      tmem_st16(tS, pk);
      tmem_st16(tS + 16, pk + 16);
      bwd_publish(bar(C::kBarP));
      if (!(ok = mbar_wait_w(bar(C::kBarDp), (uint32_t)i & 1u, s_abort, p.status) &&
                 mbar_wait_w(bar(C::kBarXFull + x), (uint32_t)(i / C::kX) & 1u, s_abort, p.status)))
        break;
      tc_fence_after();
      tmem_ld32(tP, dp);
      tmem_ld32(tP + 32, dp + 32);
      tmem_wait_ld();
      const float4* vd = reinterpret_cast<const float4*>(smem + C::kOffD + x * C::kVecBytes) + r0 / 4;
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
        const float4 d = vd[e / 4];
        pk[e / 2] = pack2<E>(s[e] * (dp[e] - d.x), s[e + 1] * (dp[e + 1] - d.y));
        pk[e / 2 + 1] = pack2<E>(s[e + 2] * (dp[e + 2] - d.z), s[e + 3] * (dp[e + 3] - d.w));
      }
      tmem_st16(tP, pk);
      tmem_st16(tP + 16, pk + 16);
      bwd_publish(bar(C::kBarDs));
    }
    if (ok && n_steps > 0) {
      ok = mbar_wait_w(bar(C::kBarDone), 0, s_abort, p.status);
      tc_fence_after();
    }
    if (ok && !FA_DBG_OK(p.status, bhk < p.B * p.H_kv && tmem_in(lane_base + C::kTmA, D) &&
                                      tmem_in(lane_base + C::kTmB, D)))
      ok = false;   // FA_DEBUG: reported; nothing stored
    if (ok) {   // warp-uniform; keys past N_k (a ragged last block) load but do not store
      const bool valid = key < p.N_k;
      if constexpr (WIN) {
        if (parts > 1) {   // warpgroup 0 holds dV, warpgroup 1 dK; a warp's 32 keys are contiguous
          const int id = (bhk * p.n_sb + kb) * parts + part;
          float4* dst = reinterpret_cast<float4*>(p.part) + ((size_t)(id * 2 + grp) * (D / 4)) * kT + k;
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            float v[32];
            if (n_steps > 0) {
              tmem_ld32(tmem + lane_base + (grp == 0 ? C::kTmA : C::kTmB) + (uint32_t)cc, v);
              tmem_wait_ld();
            }
#pragma unroll
            for (int g = 0; g < 8; ++g)
              __stcg(dst + (size_t)(cc / 4 + g) * kT,
                     n_steps > 0 ? make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3])
                                 : make_float4(0.f, 0.f, 0.f, 0.f));
          }
        }
      }
      if (!WIN || parts == 1) {   // warpgroup 0 writes dV, warpgroup 1 dK
        const size_t row = ((size_t)bhk * p.N_k + (valid ? key : 0)) * D;
        if (grp == 0)
          store_row<D, E>(tmem + lane_base + C::kTmA, static_cast<uint16_t*>(p.dv) + row, 1.f, n_steps == 0, valid);
        else
          store_row<D, E>(tmem + lane_base + C::kTmB, static_cast<uint16_t*>(p.dk) + row, p.scale, n_steps == 0,
                          valid);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kBwdWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- dQ
template <int D, Elem E, bool WIN>
__device__ __forceinline__ void bwd_dq_cta(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                           const CUtensorMap& tmdO, const BwdParams& p, int blk) {
  using C = BwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::kOffBar + 8 * i; };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int bhq = blk / p.n_qt;
  const int t = p.n_qt - 1 - (blk - bhq * p.n_qt);   // descending: under a causal mask the last tiles are the longest
  const int b = bhq / p.H_q, h = bhq - b * p.H_q;
  const int bhk = b * p.H_kv + h / p.G;
  const int q0 = t * kT;
  // key blocks seen by some row of the tile
  int n_steps = p.n_kb;
  if (p.causal) {
    const int last = min(q0 + kT - 1, p.N_q - 1) + p.kv_off;   // the last key the tile sees
    n_steps = last < 0 ? 0 : min(p.n_kb, last / kT + 1);
  }
  // WIN: the sink blocks, then the window's; step j is key block block_of(j)
  KeyTiles kt{0, 0, n_steps};
  if constexpr (WIN) {
    kt = key_tiles_of(q0 + p.kv_off, min(q0 + kT, p.N_q) + p.kv_off, p.window, p.sinks);
    n_steps = kt.count();
  }
  auto block_of = [&](int j) { return WIN ? kt.tile(j) : j; };

  // step j's tiles (FA_DEBUG: false when not in their tensors)
  auto load_x = [&](int j) {
    const int x = j % C::kX;
    if (!FA_DBG_OK(p.status, block_of(j) < p.n_kb && bhk < p.B * p.H_kv)) return false;
    mbar_arrive_expect_tx(bar(C::kBarXFull + x), C::kTileBytes);
    bwd_load_tile<D>(sb + C::kOffX + x * C::kTileBytes, tmK, bar(C::kBarXFull + x), block_of(j) * kT, bhk);
    return true;
  };
  auto load_y = [&](int j) {
    const int y = j % C::kY;
    mbar_arrive_expect_tx(bar(C::kBarYFull + y), C::kTileBytes);
    bwd_load_tile<D>(sb + C::kOffY + y * C::kTileBytes, tmV, bar(C::kBarYFull + y), block_of(j) * kT, bhk);
  };
  const uint32_t tmem = bwd_setup<D>(smem, warp, lane, [&] {
    if (n_steps == 0) return;
    const size_t vo = (size_t)bhq * p.nq_pad + q0;
    mbar_arrive_expect_tx(bar(C::kBarRes), C::kTileBytes + 2 * C::kVecBytes);
    bwd_load_tile<D>(sb + C::kOffRes, tmQ, bar(C::kBarRes), q0, bhq);
    bulk_copy_1d(sb + C::kOffLse, p.lse2 + vo, C::kVecBytes, bar(C::kBarRes));
    bulk_copy_1d(sb + C::kOffD, p.dsum + vo, C::kVecBytes, bar(C::kBarRes));
    load_x(0);
    mbar_arrive_expect_tx(bar(C::kBarRes + 1), C::kTileBytes);
    bwd_load_tile<D>(sb + C::kOffRes + C::kTileBytes, tmdO, bar(C::kBarRes + 1), q0, bhq);
    load_y(0);
  });

  if (warp == kBwdWarpProducer) {
    if (lane == 0 && n_steps > 0) {
      int nx = 1, ny = 1;
      for (int j = 1; j < n_steps; ++j) {
        const int x = j % C::kX, y = j % C::kY;
        if (!mbar_wait(bar(C::kBarXEmpty + x), ((uint32_t)(j / C::kX) & 1u) ^ 1u, s_abort, p.status)) break;
        if (!load_x(j)) break;   // reported, not loaded
        ++nx;
        if (!mbar_wait(bar(C::kBarYEmpty + y), ((uint32_t)(j / C::kY) & 1u) ^ 1u, s_abort, p.status)) break;
        load_y(j);
        ++ny;
      }
      bwd_drain_loads<D>(sb + C::kOffBar, nx, ny, p.status);
    }
    __syncwarp();
  } else if (warp == kBwdWarpMma) {
    if (n_steps > 0) bwd_mma<D, E, WIN ? Pass::kDqSum : Pass::kDq>(sb, tmem, n_steps, s_abort, p.status);
    __syncwarp();
  } else if (warp < 8) {
    // ---- element-wise: this thread is query row r of the tile (TMEM lane r),
    // in warpgroup grp, which takes the 64-key chunk grp of every block
    const int grp = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int row = q0 + r;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::kTmS + 64 * grp, tP = tmem + lane_base + C::kTmP + 64 * grp;
    const float c = p.c;
    bool ok = true;
    float l2 = INFINITY, dd = 0.f;
    if (n_steps > 0) {
      ok = mbar_wait_w(bar(C::kBarRes), 0, s_abort, p.status);
      l2 = reinterpret_cast<const float*>(smem + C::kOffLse)[r];
      dd = reinterpret_cast<const float*>(smem + C::kOffD)[r];
    }
    // keys at or past `lim` are masked (ragged key range, causal diagonal)
    const int lim = p.causal ? min(p.N_k, row + p.kv_off + 1) : p.N_k;
    // WIN: and those in [sinks, lo), before the row's window
    const int lo = WIN ? row + p.kv_off + 1 - p.window : 0;
    [[maybe_unused]] float rsum0 = 0.f, rsum1 = 0.f;   // WIN: this thread's keys' dS, summed
    for (int j = 0; j < n_steps && ok; ++j) {
      if (!(ok = mbar_wait_w(bar(C::kBarS), (uint32_t)j & 1u, s_abort, p.status))) break;
      tc_fence_after();
      const int key0 = block_of(j) * kT + 64 * grp;
      if (!FA_DBG_OK(p.status, tmem_in(lane_base + C::kTmS + 64 * grp, 64) && tmem_in(lane_base + C::kTmP + 64 * grp, 64))) {
        ok = false;   // FA_DEBUG: reported; this step is not processed
        break;
      }
      float s[64], dp[64];
      tmem_ld32(tS, s);
      tmem_ld32(tS + 32, s + 32);
      tmem_wait_ld();
      if constexpr (!WIN) {   // (no product takes P: S may be overwritten)
        tc_fence_before();
        mbar_arrive(bar(C::kBarP));
      }
      // (the mask: as in the other role)
      if (__any_sync(0xffffffffu, key0 + 64 > lim || (WIN && key0 < lo && key0 + 64 > p.sinks))) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (key0 + e >= lim || (WIN && key0 + e < lo && key0 + e >= p.sinks)) s[e] = -INFINITY;
      }
      uint32_t pk[32];
#pragma unroll
      for (int e = 0; e < 64; e += 2) {
        s[e] = ex2_approx(s[e] * c - l2);
        s[e + 1] = ex2_approx(s[e + 1] * c - l2);
        if constexpr (WIN) pk[e / 2] = pack2<E>(s[e], s[e + 1]);
      }
      if constexpr (WIN) {   // P of the chunk's 64 keys over its own first 32 columns (read above)
        tmem_st16(tS, pk);
        tmem_st16(tS + 16, pk + 16);
        bwd_publish(bar(C::kBarP));
      }
      if (!(ok = mbar_wait_w(bar(C::kBarDp), (uint32_t)j & 1u, s_abort, p.status))) break;
      tc_fence_after();
      tmem_ld32(tP, dp);
      tmem_ld32(tP + 32, dp + 32);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 64; e += 2) {
        const float d0 = s[e] * (dp[e] - dd), d1 = s[e + 1] * (dp[e + 1] - dd);
        pk[e / 2] = pack2<E>(d0, d1);
        if constexpr (WIN) {
          rsum0 += d0;
          rsum1 += d1;
        }
      }
      tmem_st16(tP, pk);
      tmem_st16(tP + 16, pk + 16);
      bwd_publish(bar(C::kBarDs));
    }
    if (ok && n_steps > 0) {
      ok = mbar_wait_w(bar(C::kBarDone), 0, s_abort, p.status);
      tc_fence_after();
    }
    if (ok && !FA_DBG_OK(p.status, bhq < p.B * p.H_q && tmem_in(lane_base + C::kTmB, D)))
      ok = false;   // FA_DEBUG: reported; nothing stored
    [[maybe_unused]] float rr = 0.f;
    if constexpr (WIN) {
      // r from both warpgroups' keys, through the resident vectors (every thread has read
      // its own at the start); all eight warps take the barriers, whatever became of ok
      float* rs = reinterpret_cast<float*>(smem + C::kOffLse);
      named_bar_sync(2, kBwdEwThreads);
      rs[grp * kT + r] = rsum0 + rsum1;
      named_bar_sync(2, kBwdEwThreads);
      rr = rs[r] + rs[kT + r];
    }
    if (ok) {   // warp-uniform; rows past N_q (a ragged last tile) load but do not store
      const bool valid = row < p.N_q;   // warpgroup g writes columns [g D/2, (g+1) D/2)
      if constexpr (WIN) {
        if (grp == 0 && valid) p.dsum[(size_t)bhq * p.nq_pad + row] = dd + rr;
        uint16_t* dst = static_cast<uint16_t*>(p.dq) + ((size_t)bhq * p.N_q + (valid ? row : 0)) * D;
#pragma unroll 1
        for (int cc = grp * (D / 2); cc < (grp + 1) * (D / 2); cc += 32) {
          float a[32], b[32];
          if (n_steps > 0) {
            tmem_ld32(tmem + lane_base + C::kTmB + (uint32_t)cc, a);
            tmem_ld32(tmem + lane_base + C::kTmA + (uint32_t)cc, b);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] = n_steps > 0 ? fmaf(-rr, b[i], a[i]) * p.scale : 0.f;
          if (!valid) continue;
#pragma unroll
          for (int g = 0; g < 4; ++g)
            st_global_v4(dst + cc + 8 * g, pack2<E>(a[8 * g], a[8 * g + 1]), pack2<E>(a[8 * g + 2], a[8 * g + 3]),
                         pack2<E>(a[8 * g + 4], a[8 * g + 5]), pack2<E>(a[8 * g + 6], a[8 * g + 7]));
        }
      } else {
        store_row<D, E>(tmem + lane_base + C::kTmB,
                        static_cast<uint16_t*>(p.dq) + ((size_t)bhq * p.N_q + (valid ? row : 0)) * D, p.scale,
                        n_steps == 0, valid, grp * (D / 2), (grp + 1) * (D / 2));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kBwdWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// One launch for both halves of the work: first the dK/dV CTAs of all KV heads, then the
// dQ CTAs, so that the second role fills the SMs that the first one's tail leaves. Within
// a role the KV heads follow each other, and in a head the longest work goes first (key
// blocks ascending, query tiles descending: under a causal mask those are the long ones),
// the group's query heads interleaved. (A head's dK/dV CTAs followed by its dQ CTAs keeps
// its tiles in L2 for both, but then the grid ends with a head's long dK/dV CTAs: causal,
// 32 heads x 4096 rows 502 us against 402, 32/8 heads 545 against 360, without the mask
// 672 against 656.)
// How the two roles share launches: both in one grid, or (under a window) one each.
enum class Roles : int { kBoth = 0, kWindowDq = 1, kWindowDkDv = 2 };
template <int D, Elem E, Roles W>
__global__ void __launch_bounds__(kBwdThreads, 1)
    fa_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                  const BwdParams p) {
  if constexpr (W == Roles::kWindowDkDv) {   // the sink blocks of every KV head first
    const int n = p.B * p.H_kv * p.n_sb * p.sink_parts;
    const bool sink = (int)blockIdx.x < n;
    const int parts = sink ? p.sink_parts : 1, per = sink ? p.n_sb * parts : p.n_kb - p.n_sb;
    const int cta = (int)blockIdx.x - (sink ? 0 : n);
    const int bhk = cta / per, w = cta - bhk * per;
    bwd_dkdv_cta<D, E, true>(tmQ, tmK, tmV, tmdO, p, bhk, sink ? w / parts : p.n_sb + w, sink ? w % parts : 0, parts);
    return;
  }
  constexpr bool kDqOnly = W == Roles::kWindowDq;
  int cta = (int)blockIdx.x;
  if constexpr (!kDqOnly) {
    const int n = p.B * p.H_kv * p.n_kb;
    if (cta < n) {
      const int bhk = cta / p.n_kb;
      bwd_dkdv_cta<D, E, false>(tmQ, tmK, tmV, tmdO, p, bhk, cta - bhk * p.n_kb);
      return;
    }
    cta -= n;
  }
  // rank idx / G of query head G * (KV head) + idx % G
  const int bhk = cta / (p.G * p.n_qt), idx = cta - bhk * (p.G * p.n_qt);
  const int rank = idx / p.G, gi = idx - rank * p.G;
  bwd_dq_cta<D, E, kDqOnly>(tmQ, tmK, tmV, tmdO, p, (bhk * p.G + gi) * p.n_qt + rank);
}

// dK and dV of the sink blocks: the parts' sums, in order. One block of 128 threads (keys)
// per (KV head, sink block), 8 columns and gradient.
template <int D, Elem E>
__global__ void __launch_bounds__(kT) fa_bwd_sink_kernel(const BwdParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int k = threadIdx.x, c8 = blockIdx.y >> 1, which = blockIdx.y & 1;   // 0: dV, 1: dK
  const int bhk = blockIdx.x / p.n_sb, kb = blockIdx.x - bhk * p.n_sb;
  const int key = kb * kT + k;
  if (key >= p.N_k) return;
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = 0.f;
#pragma unroll 4
  for (int x = 0; x < p.sink_parts; ++x) {
    const float4* src = reinterpret_cast<const float4*>(p.part) +
                        ((size_t)((blockIdx.x * p.sink_parts + x) * 2 + which) * (D / 4) + 2 * c8) * kT + k;
    const float4 u = __ldcg(src), v = __ldcg(src + kT);
    a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
    a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
  }
  const float m = which == 0 ? 1.f : p.scale;
  st_global_v4(static_cast<uint16_t*>(which == 0 ? p.dv : p.dk) + ((size_t)bhk * p.N_k + key) * D + 8 * c8,
               pack2<E>(a[0] * m, a[1] * m), pack2<E>(a[2] * m, a[3] * m), pack2<E>(a[4] * m, a[5] * m),
               pack2<E>(a[6] * m, a[7] * m));
}

// A launch whose kernel may set itself up while the one before it on the stream ends, and
// waits for it then (griddepcontrol.wait). The window's kernels after the first are launched
// so, each waiting for all before it: 1000 rows 32.7 -> 30.4 us, 8192 rows 528 -> 526. With
// both roles in one grid it costs (one head, 8192 rows: 101 -> 118 us; the CTAs that start
// during the first kernel lie unevenly), so that launch is an ordinary one.
template <typename... K, typename... A>
cudaError_t launch_after(void (*kernel)(K...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <int D, Elem E, Roles W>
cudaError_t launch_bwd_main_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const BwdParams& p, int ctas, cudaStream_t stream) {
  using C = BwdCfg<D>;
  static bool attr[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!attr[dev]) {
    cudaError_t e = cudaFuncSetAttribute(fa_bwd_kernel<D, E, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::kLaunchSmem);
    if (e != cudaSuccess) return e;
    attr[dev] = true;
  }
  if constexpr (W == Roles::kBoth)
    return launch_kernel(fa_bwd_kernel<D, E, W>, dim3((unsigned)ctas), dim3(kBwdThreads), C::kLaunchSmem, stream, tq,
                         tk, tv, tdo, p);
  return launch_after(fa_bwd_kernel<D, E, W>, dim3((unsigned)ctas), dim3(kBwdThreads), C::kLaunchSmem, stream, tq, tk,
                      tv, tdo, p);
}

template <int D, Elem E>
cudaError_t launch_bwd_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                         const CUtensorMap& tdo, const BwdParams& p, const void* o, const void* dout,
                         const float* lse, float* lse2, float* dsum, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.H_q * p.nq_pad;
  cudaError_t e = launch_kernel(fa_bwd_prep_kernel<D, E>, dim3((unsigned)((rows + 8 * kPrepRows - 1) / (8 * kPrepRows))), dim3(256), 0,
                                stream, static_cast<const uint16_t*>(o), static_cast<const uint16_t*>(dout), lse, lse2,
                                dsum, p.N_q, p.nq_pad, rows);
  if (e != cudaSuccess) return e;
  const int dkdv = p.B * p.H_kv * p.n_kb, dq = p.B * p.H_q * p.n_qt;
  if (p.window == 0) return launch_bwd_main_t<D, E, Roles::kBoth>(tq, tk, tv, tdo, p, dkdv + dq, stream);
  e = launch_bwd_main_t<D, E, Roles::kWindowDq>(tq, tk, tv, tdo, p, dq, stream);
  if (e != cudaSuccess) return e;
  const int sinks = p.B * p.H_kv * p.n_sb;
  e = launch_bwd_main_t<D, E, Roles::kWindowDkDv>(tq, tk, tv, tdo, p, dkdv + sinks * (p.sink_parts - 1), stream);
  if (e != cudaSuccess || p.sink_parts == 1) return e;
  return launch_after(fa_bwd_sink_kernel<D, E>, dim3((unsigned)sinks, D / 8 * 2), dim3(kT), 0, stream, p);
}

bool aligned16p(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return na && nb && a0 < b0 + nb && b0 < a0 + na;
}

int backward_impl(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dout,
                  void* dq, void* dk, void* dv, int B, int H_q, int H_kv, int N_q, int N_k, int d, int causal,
                  float scale, int elem, cudaStream_t strm, int window = 0, int sinks = 0) {
  const Shape s{B, H_q, H_kv, N_q, N_k, d};
  int st = validate_shape(s);
  if (st != FA_OK) return st;
  if (d == 256) return FA_ERR_UNSUPPORTED;   // the backward kernels cover d = 64 and 128
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  const long long rows_q = (long long)B * H_q * N_q, rows_k = (long long)B * H_kv * N_k;
  const size_t qb = (size_t)rows_q * d * 2, kb = (size_t)rows_k * d * 2;
  const void* ins[6] = {q, k, v, o, lse, dout};
  const size_t in_bytes[6] = {qb, kb, kb, qb, (size_t)rows_q * 4, qb};
  void* outs[3] = {dq, dk, dv};
  const size_t out_bytes[3] = {qb, kb, kb};
  for (int i = 0; i < 6; ++i)
    if (in_bytes[i] && (!ins[i] || !aligned16p(ins[i]))) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (out_bytes[i] && (!outs[i] || !aligned16p(outs[i]))) return FA_ERR_INVALID_ARG;
    for (int j = 0; j < 6; ++j)
      if (overlap(outs[i], out_bytes[i], ins[j], in_bytes[j])) return FA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], out_bytes[i], outs[j], out_bytes[j])) return FA_ERR_INVALID_ARG;
  }
  {
    const void* all[9];
    for (int i = 0; i < 6; ++i) all[i] = in_bytes[i] ? ins[i] : nullptr;
    for (int i = 0; i < 3; ++i) all[6 + i] = out_bytes[i] ? outs[i] : nullptr;
    st = check_current_device(all, 9);
    if (st != FA_OK) return st;
  }
  // nothing to differentiate through: every gradient that exists is zero
  if (rows_q == 0 || rows_k == 0) {
    for (int i = 0; i < 3; ++i) {
      if (!out_bytes[i]) continue;
      cudaError_t e = cudaMemsetAsync(outs[i], 0, out_bytes[i], strm);
      if (e != cudaSuccess) return cuda_fail(e);
    }
    return FA_OK;
  }
  int* status = device_status_ptr();
  if (!status) return cuda_fail(cudaGetLastError());
  BwdParams p{};
  p.B = B; p.H_q = H_q; p.H_kv = H_kv; p.N_q = N_q; p.N_k = N_k; p.G = H_q / H_kv;
  p.causal = causal ? 1 : 0;
  p.kv_off = N_k - N_q;
  p.n_qt = (N_q + kT - 1) / kT;
  p.n_kb = (N_k + kT - 1) / kT;
  p.nq_pad = p.n_qt * kT;
  // a window over every key leaves nothing to the sinks
  p.window = window < N_k ? window : (window > 0 ? N_k : 0);
  p.sinks = window < N_k ? sinks : 0;
  if (p.sinks > N_k) p.sinks = N_k;
  p.n_sb = p.window > 0 ? (p.sinks + kT - 1) / kT : 0;
  p.c = scale * kLog2e;
  p.scale = scale;
  p.dq = dq; p.dk = dk; p.dv = dv;
  p.status = status;
  if ((long long)B * H_q * p.n_qt + (long long)B * H_kv * p.n_kb >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  CUtensorMap tq, tk, tv, tdo;
  if (!make_tmap_bf16_3d(&tq, q, d, N_q, (uint64_t)B * H_q, d, kT) ||
      !make_tmap_bf16_3d(&tdo, dout, d, N_q, (uint64_t)B * H_q, d, kT) ||
      !make_tmap_bf16_3d(&tk, k, d, N_k, (uint64_t)B * H_kv, d, kT) ||
      !make_tmap_bf16_3d(&tv, v, d, N_k, (uint64_t)B * H_kv, d, kT))
    return cuda_fail(cudaErrorInvalidValue);
  // sink blocks: cut so that no part is longer than half an even share of all steps
  // (two CTAs an SM's worth), or than 8 steps
  size_t part_bytes = 0;
  p.sink_parts = 1;
  if (p.n_sb > 0) {
    const long long reach = (p.window + 2ll * kT - 2) / kT + 1;   // query tiles that see a block, at most
    const long long steps = (long long)B * H_q * (p.n_sb * (long long)p.n_qt + (p.n_kb - p.n_sb) *
                                                  (reach < p.n_qt ? reach : (long long)p.n_qt));
    const long long share = steps / (2ll * num_sms()), most = share > 8 ? share : 8;
    const long long parts = ((long long)p.G * p.n_qt + most - 1) / most;
    p.sink_parts = (int)(parts < 64 ? parts : 64);
    if (p.sink_parts > 1) part_bytes = (size_t)B * H_kv * p.n_sb * p.sink_parts * 2 * kT * d * 4;
  }
  const WorkspaceSource& pool = pool_workspace();
  const size_t vec = (size_t)B * H_q * p.nq_pad * 4;
  void* ws = nullptr;
  st = pool.acquire(2 * vec + part_bytes, strm, &ws);
  if (st != FA_OK) return st;
  float* lse2 = static_cast<float*>(ws);
  float* dsum = reinterpret_cast<float*>(static_cast<char*>(ws) + vec);
  p.lse2 = lse2;
  p.dsum = dsum;
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * vec);
  cudaError_t e;
  if (elem == (int)Elem::F16)
    e = d == 128 ? launch_bwd_t<128, Elem::F16>(tq, tk, tv, tdo, p, o, dout, lse, lse2, dsum, strm)
                 : launch_bwd_t<64, Elem::F16>(tq, tk, tv, tdo, p, o, dout, lse, lse2, dsum, strm);
  else
    e = d == 128 ? launch_bwd_t<128, Elem::BF16>(tq, tk, tv, tdo, p, o, dout, lse, lse2, dsum, strm)
                 : launch_bwd_t<64, Elem::BF16>(tq, tk, tv, tdo, p, o, dout, lse, lse2, dsum, strm);
  if (pool.release) pool.release(ws, strm);
  return e == cudaSuccess ? FA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace fa

extern "C" int fa_backward(const void* q, const void* k, const void* v, const void* o, const float* lse,
                           const void* dout, void* dq, void* dk, void* dv, int B, int H_q, int H_kv, int N_q,
                           int N_k, int d, int causal, float scale, int dtype, void* stream) {
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_INVALID_ARG;
  return fa::backward_impl(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d, causal, scale, dtype,
                           static_cast<cudaStream_t>(stream));
}

extern "C" int fa_backward_window(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                  const void* dout, void* dq, void* dk, void* dv, int B, int H_q, int H_kv, int N_q,
                                  int N_k, int d, int window, int sinks, float scale, int dtype, void* stream) {
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_FP16) return FA_ERR_INVALID_ARG;
  if (window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  return fa::backward_impl(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d, 1, scale, dtype,
                           static_cast<cudaStream_t>(stream), window, sinks);
}
