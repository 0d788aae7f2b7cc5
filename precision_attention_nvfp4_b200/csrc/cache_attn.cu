// Attention over the paged FP8 KV cache.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i)
// over the cached tokens j that query i sees; lse_i = m_i + log sum_j p_ij.
//
// A step of a served model reads every cached byte once for a handful of
// query rows, so the products are laid out with the keys, not the queries, on
// the tensor core's 128 rows: S^T = K Q^T has 128 keys by N query rows, O^T =
// V^T P^T has d channels by N query rows (N = 16 or 32: the queries and heads that
// share a KV head; for more rows see the kernel further down). K and V go from the
// cache to the MMA as they are, E4M3 bytes moved by TMA; nothing is converted on the way. What
// has to stay precise is split instead, at N rows it is nearly free:
//   Q = Qhi + Qlo, both E4M3 at a power-of-two scale a row: the 8 bits of a
//     bf16 value exactly, to 2^-10 of a scale that brings the row to 224..448;
//     both products go to one accumulator
//   P = P1 + 2^-3 P2 + 2^-7 P3, all E5M2 (3 bits each): 2^-9 of the value. The terms lie side
//     by side in 3 N columns of one product, which reads V once, into three
//     accumulators that are added at the end
// The rows' scales are powers of two: K's multiplies its scores, V's is added to the
// exponent of P, so that P V needs no scale, and taken out of the row sum. So what is split
// is P 2^ev, 2^10 or more for the row's largest: 2^-9 of it down to 2^-24 of the largest,
// below that an error of at most 2^-33 of the largest.
//
// CTA (persistent, one an SM, 640 threads):
//   warps 0, 3   TMA: K, and V with the scales, in 128-key tiles into two rings, page by page
//   warp 1       issues O^T += V^T P^T (one thread); owns tensor memory
//   warp 2       issues S^T = K Q^T (one thread)
//   warps 4-19   four softmax warpgroups, one key a thread: two take the tiles in
//                turn for each half of the query rows (or four take them in
//                turn), with their own reference maxima, row sums and O, so that
//                none waits on another; joined at a segment's end. They also
//                load, scale and split the query rows of the next segment
// The reference maximum of a row moves only when P would pass E5M2's largest,
// and P is 2^10 then, so that it seldom moves again; the 128
// threads of a warpgroup agree on it with one barrier a group of rows, and O in
// tensor memory is rescaled only then.
//
// Work: the tiles of all (sequence, row tile, KV head) problems form one list
// that is cut evenly over the CTAs, so mixed lengths balance and a single long
// sequence fills the card. A CTA's piece of a problem is a segment; a problem
// cut in several leaves unnormalised partial results in the workspace, which
// a second launch joins in a fixed order (no atomics: repeats are bit-identical).
//
// Bound by reading the cache where there are few rows: 64 sequences of 16384 tokens
// at most, 8 heads of 128 channels, 1.1 GB: 174 us, 6.3 TB/s, among passes over other
// caches; 198 us, 5.5 TB/s, behind a pass that leaves L2 full of written lines. One
// sequence of 131072 tokens 55 us, 4.9 TB/s, of which 12 us are the two launches,
// planning and the join.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fpattn_internal.h"
#include "serve_internal.h"
#include "sm100.cuh"

namespace fpattn {

namespace {

__device__ int g_cache_attn_error = 0;

constexpr int kSegs = 64;           // segments a CTA plans at a time
// What a problem costs besides its tiles, in tiles: its rows are loaded and split, its results joined and stored.
// 64 sequences of up to 16384 tokens, one query each (8 KV heads, group 4): 224 us at 0, 188 at 4, 174 at 8, 177 at 12,
// 178 at 16; d = 64: 199, 170, 146, 148, 151; of up to 2048 tokens (d = 128): 108, 59, 47, 49, 50. Tiles of 128 rows
// (3 chunks of up to 1024 queries, d = 128): 532 us at 2, 506 at 4, 493 at 6, 498 at 8, 508 at 12.
template <int N>
constexpr int kSegCost = N == 128 ? 6 : 8;
// A P above 2^kPTop moves the reference maximum, and is 2^kPLog2 then: the further apart, the less often, and the less of
// P's range lies below. (Trees of 8 tokens on 8 sequences of up to 16384, 32 rows a KV head: 61 us with 13, 49 with 10,
// 48 with 7; 64 sequences of up to 2048, one token: 50, 47 and 47; chunks of many rows, d = 128: 536, 493 and 484.)
// kPTop is below the largest E5M2 (57344) and fp16.
constexpr float kPLog2 = 10.f;
constexpr float kPTop = 15.75f;
// What P1 leaves is at most 2^12, what P2 leaves of that 2^8: scaled into E5M2's range, the terms reach further down.
constexpr float kMidScale = 8.f, kLoScale = 128.f;
constexpr float kNever = -3e38f;    // reference maximum before any key was seen: below every score
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

// which bounded wait gave up
enum : int {
  kErrKEmpty = 0x1101, kErrKFull = 0x1102, kErrVFull = 0x1103, kErrQFull = 0x1104,
  kErrSFull = 0x1106, kErrSFree = 0x1107, kErrPFull = 0x1108, kErrODone = 0x1109, kErrEpi = 0x110a, kErrDrain = 0x110b,
  kErrVEmpty = 0x110c, kErrScales = 0x110d
};

// ---------------------------------------------------------------------------
// Instructions
// ---------------------------------------------------------------------------
// Descriptor with F32 accumulate; type 0: E4M3 of kind::f8f6f4, fp16 of kind::f16, 1: E5M2. major 1: MN.
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn, int b_type = 0) {
  return (1u << 4) | (static_cast<uint32_t>(b_type) << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t swz_of(int row_bytes) { return row_bytes == 128 ? 2u : (row_bytes == 64 ? 4u : 6u); }
// 16-byte chunks of a row permuted as the 128-, 64- or 32-byte swizzle does.
template <int kRow>
__device__ __forceinline__ uint32_t swizzled(uint32_t off) {
  return off ^ (((off >> 7) & (kRow / 16 - 1)) << 4);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 8 or 16 columns, waited for: one block, so that the results need no copies.
template <int kRegs>
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t* r) {
  if (kRegs == 8)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
template <int kRegs>
__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t* r) {
  if (kRegs == 8)
    tmem_st8(taddr, r);
  else
    tmem_st16(taddr, reinterpret_cast<const uint32_t(&)[16]>(*r));
}
__device__ __forceinline__ void tmem_wait8(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
// One page of one head, at coordinates (0, 0, page * H + head).
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int ph) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(ph)
      : "memory");
}
__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// D[tmem] (+)= A[tmem] * B[smem], kind::f16 (fp16 x fp16 -> F32); A is K-major in TMEM, two values a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// What is to be added to a row's exponents instead of nb, so that the largest, now `top`, becomes kPLog2. (For scores of
// 2^27 and more a step of the sum is as large as P's range: then one that does not carry P past its largest.)
__device__ __forceinline__ float reference(float top, float nb) {
  const float now = nb + (kPLog2 - top);
  return top + (now - nb) > kPTop ? now - fabsf(now) * 1.1920929e-7f : now;
}
// Both no more than top; a NaN stays.
__device__ __forceinline__ uint64_t at_most(uint64_t x, float top) {
  float a, b;
  f2_unpack(x, a, b);
  return f2_pack(a > top ? top : a, b > top ? top : b);
}
// Barrier of `n` threads; every thread of them always takes part (see the loops).
__device__ __forceinline__ void named_sync(int id, int n) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ bool named_any(int id, int n, bool x) {
  uint32_t y;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(id), "r"(n), "r"(x ? 1u : 0u)
      : "memory");
  return y != 0;
}
// Four P as three E5M2 codes each: hi + mid / kMidScale + lo / kLoScale. (E5M2 is fp16's upper byte, so what a term
// leaves is exact in fp16. One block: the 16-bit halves are then packed by the conversions themselves.)
__device__ __forceinline__ void split_p(float p0, float p1, float p2, float p3, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  asm("{\n\t"
      ".reg .b16 a, b;\n\t"
      ".reg .b32 h0, h1, r0, r1;\n\t"
      "cvt.rn.f16x2.f32 h0, %4, %3;\n\t"
      "cvt.rn.f16x2.f32 h1, %6, %5;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 a, h0;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 b, h1;\n\t"
      "mov.b32 %0, {a, b};\n\t"
      "prmt.b32 r0, %0, 0, 0x1404;\n\t"
      "prmt.b32 r1, %0, 0, 0x3424;\n\t"
      "sub.rn.f16x2 h0, h0, r0;\n\t"
      "sub.rn.f16x2 h1, h1, r1;\n\t"
      "mul.rn.f16x2 h0, h0, %7;\n\t"
      "mul.rn.f16x2 h1, h1, %7;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 a, h0;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 b, h1;\n\t"
      "mov.b32 %1, {a, b};\n\t"
      "prmt.b32 r0, %1, 0, 0x1404;\n\t"
      "prmt.b32 r1, %1, 0, 0x3424;\n\t"
      "sub.rn.f16x2 h0, h0, r0;\n\t"
      "sub.rn.f16x2 h1, h1, r1;\n\t"
      "mul.rn.f16x2 h0, h0, %8;\n\t"
      "mul.rn.f16x2 h1, h1, %8;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 a, h0;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 b, h1;\n\t"
      "mov.b32 %2, {a, b};\n\t}"
      : "=&r"(hi), "=&r"(mid), "=r"(lo)
      : "f"(p0), "f"(p1), "f"(p2), "f"(p3), "r"(0x48004800u), "r"(0x4C004C00u));  // twice 8, kMidScale; 16, the rest
}
// Two P as packed fp16.
__device__ __forceinline__ uint32_t half_p(float p0, float p1) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(h) : "f"(p0), "f"(p1));
  return h;
}
// Four E4M3 codes as fp16 (exact).
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
  uint2 h;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h.x), "=r"(h.y)
      : "r"(codes));
  return h;
}
// A key's V row from the tile as TMA laid it out to a tile of fp16: [64 channels][128 keys][128 bytes], 128-byte swizzle.
// Zeros where the key is not there: what lies behind a sequence, or in a page that is not there, may be NaN, and
// 0 * NaN would reach O. (Eight lanes take eight keys' same 16 channels: no bank conflicts on either side.)
template <int D, int kChunks>
__device__ __forceinline__ void widen_row(const uint8_t* tile, uint8_t* wide, int key, int c0, bool live) {
  const uint32_t keep = live ? ~0u : 0u;
  uint4 x[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) x[c] = *reinterpret_cast<const uint4*>(tile + swizzled<D>(key * D + (c0 + c) * 16));
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint2 a = widen4(x[c].x & keep), b = widen4(x[c].y & keep), e = widen4(x[c].z & keep), f = widen4(x[c].w & keep);
    uint8_t* dst = wide + ((c0 + c) / 4) * 128 * 128;
    *reinterpret_cast<uint4*>(dst + swizzled<128>(key * 128 + ((c0 + c) % 4) * 32)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4*>(dst + swizzled<128>(key * 128 + ((c0 + c) % 4) * 32 + 16)) = make_uint4(e.x, e.y, f.x, f.y);
  }
}

// ---------------------------------------------------------------------------
// Layout
// ---------------------------------------------------------------------------
// One CTA's piece of a problem: tiles j0 .. j0 + nt - 1 of the keys of
// sequence b and KV head h, for query rows rt * N .. of its T * group rows.
struct Seg {
  int b, h, rt, j0, nt, row0, T, L, slot;  // row0: first row of q; slot: of the workspace, -1: results go out
};

template <int D, int N>
struct Cfg {
  static constexpr int kD = D, kThreads = 640;
  static constexpr int kTile = 128 * D;                    // bytes of a K or V tile
  // The four softmax warpgroups: kPar of them take the tiles in turn, kHalves share a tile's query rows. A tile of 16
  // rows and 64 channels is little work behind a long chain of waits, so more of them go at once (batch of 64 at 16384
  // tokens: 146 us with four and one, 152 with two and two; at 128 channels 178 and 174, one sequence of 131072 57
  // and 55, 64 of up to 2048 50 and 47).
  static constexpr int kPar = N == 16 && D == 64 ? 4 : 2, kHalves = 4 / kPar;
  static constexpr int kPP = 4 * N;                        // row pitch of a P tile: a key's three terms, N bytes each
  static constexpr int kPTile = 128 * kPP;
  static constexpr int kQ = N * D;                         // bytes of one term of Q
  static constexpr int kFixed = 2 * 2 * kQ + kPar * kPTile + 1024 * 8;
  static constexpr int kRoom = (227 * 1024 - 1024 - kFixed) / (2 * kTile + 256);
  static constexpr int kStages = kRoom > 14 ? 14 : kRoom;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffQ = kOffV + kStages * kTile;    // [2 buffers][2 terms][N][D]
  static constexpr int kOffP = kOffQ + 4 * kQ;             // [kPar][128 keys][3 terms][N]
  static constexpr int kOffE = kOffP + kPar * kPTile;      // [stage][pages of the tile][2][page]: scales
  static constexpr int kOffSeg = kOffE + kStages * 256;
  static constexpr int kOffF = kOffSeg + kSegs * static_cast<int>(sizeof(Seg));
  // 4-byte words: qmul [2][N], nbias [2 segments][kPar][N], wmax [kPar][4][N], lsum [2 segments][kPar][4][N],
  // fin [kPar + 1][N], alpha [kPar][N], lim [2][N], win [kPar][4][N]
  static constexpr int kFloats = N * (2 + 2 * kPar + 4 * kPar + 8 * kPar + kPar + 1 + kPar + 2 + 4 * kPar);
  static constexpr int kOffBias = kOffF + 4 * 2 * N, kOffMax = kOffBias + 4 * 2 * kPar * N;
  static constexpr int kOffAlpha = kOffMax + 4 * 4 * kPar * N + 4 * 8 * kPar * N + 4 * (kPar + 1) * N;
  static constexpr int kOffWin = kOffAlpha + 4 * kPar * N + 4 * 2 * N;
  static constexpr int kOffBar = (kOffF + 4 * kFloats + 7) & ~7;
  static constexpr int kBars = 4 * kStages + 4 * kPar + 2 + 1 + 2;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kOffScan = kOffMisc + 64;           // ints: units and problems of every thread's entries
  static constexpr int kBytes = kOffScan + 2 * 32 * 4 + 4 * kStages;
  static constexpr int kSmem = kBytes + 1024;
  static_assert(kSmem <= 227 * 1024 && kStages >= 3 && kStages >= kPar, "shared memory");
  // tensor memory: S [kPar][N], O [kPar][3 terms][N], row sums of every lane's keys [kPar][N]
  static constexpr int kColS = 0, kColO = kPar * N, kColL = 4 * kPar * N;
  static constexpr int kCols = 8 * kPar * N;
  static constexpr int kHalf = N / kHalves;                     // query rows of a softmax warpgroup
  static constexpr int kGroup = N == 16 ? 8 : 16;   // of them, held by a thread at once
};

struct __align__(64) Params {
  CUtensorMap tm_k, tm_v;
  CacheAttnArgs a;
  int group, RT, E;        // query heads a KV head; row tiles of the most queries; B * RT
  float scale_log2;
  int* tails;              // workspace: [CTA][8]
  float* part_ml;          // [2 CTA][2][N]
  float* part_o;           // [2 CTA][N][D]; [2 CTA][D / 4][N][4] where N is 128, whose threads hold whole rows
};

// Queries and tiles of entry e = b * RT + rt. nt 0: no such rows.
struct Entry {
  int b, rt, row0, T, L, nt;
};
template <int N>
__device__ __forceinline__ Entry entry_of(const Params& p, int e) {
  Entry r;
  r.b = e / p.RT;
  r.rt = e - r.b * p.RT;
  if (p.a.q_start) {
    r.row0 = min(max(p.a.q_start[r.b], 0), p.a.rows_total);
    r.T = min(p.a.q_start[r.b + 1], p.a.rows_total) - r.row0;  // (past Tmax: whole row tiles may be left out, not moved)
  } else {
    r.row0 = r.b * p.a.Tmax;
    r.T = p.a.Tmax;
  }
  const int cap = p.a.max_pages * p.a.cache.page_size;
  r.L = min(max(p.a.lengths[r.b], 0), cap);
  const int rows = max(r.T, 0) * p.group;
  if (r.rt * N >= rows) {
    r.nt = 0;
    return r;
  }
  int seen = r.L;  // keys any of the rows may see
  if (p.a.causal && !p.a.tree) seen = min(seen, r.L - r.T + min(rows - 1, (r.rt + 1) * N - 1) / p.group + 1);
  r.nt = max(1, (seen + 127) / 128);
  return r;
}

// One role's bounded waits: after one has failed the others return at once. A
// thread that waits is suspended for up to kNapNs at a time, so that roles with
// nothing to do leave the issue slots to the softmax warps. (How long does not show: 0, 1000 and 200000 measure the
// same within 0.5 us on batches, trees and chunks.)
constexpr uint32_t kNapNs = 20000;
__device__ __forceinline__ bool try_wait(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity), "r"(kNapNs)
      : "memory");
  return ok != 0;
}
// kCall: the slow path is a call, so that it takes no room where warps are many; not in a kernel that moves registers
// between its warps, whose calls would fix their number.
template <bool kCall>
struct Waiter {
  volatile int* abort;
  bool dead = false;
  // A whole warp waits. (A wait that is over at once costs a few instructions; a dead role's cost a nap at most.)
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity, int code) {
    const bool ok = try_wait(smem_u32(bar), parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    return kCall ? called(smem_u32(bar), parity, code) : slow(smem_u32(bar), parity, code);
  }
  __device__ __noinline__ bool called(uint32_t addr, uint32_t parity, int code) { return slow(addr, parity, code); }
  __device__ __forceinline__ bool slow(uint32_t addr, uint32_t parity, int code) {
    if (dead) return false;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
      if (__all_sync(0xffffffffu, try_wait(addr, parity))) return true;
      const bool late = globaltimer_ns() - t0 > kWaitTimeoutNs;
      if (late) {
        atomicCAS(&g_cache_attn_error, 0, code);
        *abort = 1;
      }
      if (__any_sync(0xffffffffu, late || *abort)) {
        dead = true;
        return false;
      }
    }
  }
};

// The warp's arrival, once all its lanes are past this point.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(threadIdx.x & 31)
      : "memory");
}

// The raw bytes of a segment's query rows on their way into a Q buffer: the
// first half of a row's bytes into the row of its first term, the rest into the
// second's. Warp x of the kWarps softmax warps takes rows x * kRows + sub and every
// kWarps * kRows after them; what a thread loads here it splits in split_rows.
template <int D, int N, int kWarps>
__device__ __forceinline__ void load_rows(const Params& p, const Seg& s, uint8_t* dst, int x, int lane) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int c = lane % kLanes, rows = min(N, s.T * p.group - s.rt * N);
  const int raw = (c < kLanes / 2 ? 0 : N * D) + (c % (kLanes / 2)) * 16;
  const __nv_bfloat16* q =
      static_cast<const __nv_bfloat16*>(p.a.q) + (p.a.q_start ? s.row0 * p.a.q_st : s.b * p.a.q_sb) + c * 8;
#pragma unroll 1
  for (int r = x * kRows + lane / kLanes; r < rows; r += kWarps * kRows) {
    const int t = (s.rt * N + r) / p.group, hq = s.h * p.group + (s.rt * N + r) - t * p.group;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + r * D + raw)),
                 "l"(q + t * p.a.q_st + hq * p.a.q_sh)
                 : "memory");
  }
}

// Scales those rows and splits them in place; qmul: what a row's scores are
// multiplied with, lim: the last key it sees (a tree's rows: their words say).
template <int D, int N, int kWarps>
__device__ __forceinline__ void split_rows(const Params& p, const Seg& s, uint8_t* dst, float* qmul, int* lim, int x,
                                           int lane) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const int c = lane % kLanes, sub = lane / kLanes, rows = min(N, s.T * p.group - s.rt * N);
  const int raw = (c < kLanes / 2 ? 0 : N * D) + (c % (kLanes / 2)) * 16;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll 1
  for (int r = x * kRows + sub; r < N; r += kWarps * kRows) {
    // rows that are not there see nothing, and whatever their terms hold counts nowhere
    if (c == 0) lim[r] = r >= rows ? -1 : (p.a.causal ? s.L - s.T + (s.rt * N + r) / p.group : s.L - 1);
    if (c == 0 && r >= rows) qmul[r] = 0.f;
    if (r - sub >= rows) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(dst + r * D + raw);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
    uint32_t a = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      a = max(a, max(__float_as_uint(f[2 * k]) & 0x7FFFFFFFu, __float_as_uint(f[2 * k + 1]) & 0x7FFFFFFFu));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    // the smallest e >= -100 with amax <= 448 * 2^e
    const int e = max(-100, static_cast<int>((a + 0x1FFFFFu) >> 23) - 135);
    const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x0 = f[2 * k] * up, x1 = f[2 * k + 1] * up;
      hi[k] = cvt_e4m3x2(x0, x1);
      lo[k] = cvt_e4m3x2(x0 - e4m3_to_float(hi[k]), x1 - e4m3_to_float(hi[k] >> 8));
    }
    __syncwarp();  // the rows' raw bytes were read
    const uint32_t off = swizzled<D>(r * D + c * 8);
    *reinterpret_cast<uint2*>(dst + off) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *reinterpret_cast<uint2*>(dst + N * D + off) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    // a row with a NaN or an infinity gives NaN scores
    if (c == 0 && r < rows)
      qmul[r] = a >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                                 : __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2;
  }
  fence_proxy_async_shared();
}

// Moves the references of rows c0 .. c0 + kG - 1 of a tile (parity w, called by
// the 128 threads of a warpgroup) where a score passed them: those rows take the
// tile's maximum, and their sums and O (when there is one)
// are rescaled. Out of line: few tiles need it, and its registers would crowd
// the common path's (752 instead of 579 instructions a warp and tile).
template <int D, int N>
__device__ __noinline__ void move_references(uint8_t* smem, uint32_t tmem, int c0, int wg, int buf, float km, float evf,
                                             uint32_t bit, bool masked, bool has_o) {
  using C = Cfg<D, N>;
  constexpr int kG = C::kGroup;
  const int w = wg % C::kPar, lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3, tid = q4 * 32 + lane;
  float* qm = reinterpret_cast<float*>(smem + C::kOffF) + buf * N;
  float* nb = reinterpret_cast<float*>(smem + C::kOffBias) + (buf * C::kPar + w) * N;
  float* wm = reinterpret_cast<float*>(smem + C::kOffMax) + w * 4 * N;
  float* al = reinterpret_cast<float*>(smem + C::kOffAlpha) + w * N;
  const uint32_t* seen = reinterpret_cast<const uint32_t*>(smem + C::kOffWin) + (w * 4 + q4) * N;
  const uint32_t at0 = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
  uint32_t r[kG];
  tmem_get<kG>(at0 + C::kColS + w * N + c0, r);
  float best = 0.f;
#pragma unroll
  for (int c = 0; c < kG; ++c) {
    // the exponent without the old reference, in which a first score may have been lost
    float t = fmaf(__uint_as_float(r[c]) * qm[c0 + c], km, evf);
    if (masked && !(seen[c0 + c] & bit)) t = -INFINITY;
    const float m = redux_max(t);
    if (lane == c) best = m;
  }
  if (lane < kG) wm[q4 * N + c0 + lane] = best;
  named_sync(1 + wg, 128);
  if (tid < kG) {
    const float* m4 = wm + c0 + tid;
    const float m = fmaxf(fmaxf(m4[0], m4[N]), fmaxf(m4[2 * N], m4[3 * N]));
    const float old = nb[c0 + tid], now = m + old > kPTop ? kPLog2 - m : old;
    nb[c0 + tid] = now;
    al[c0 + tid] = ex2_approx(now - old);
  }
  named_sync(1 + wg, 128);
  if (!has_o) return;
  tc_fence_after();
#pragma unroll 1
  for (int c = c0; c < c0 + kG; c += 8) {
    const float4 a = *reinterpret_cast<const float4*>(al + c), b = *reinterpret_cast<const float4*>(al + c + 4);
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    bool any = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) any = any || f[k] != 1.f;
    if (!any) continue;
#pragma unroll 1
    for (int z = 0; z < 4; ++z) {  // O's three terms, row sums
      const uint32_t at = at0 + (z < 3 ? C::kColO + (w * 3 + z) * N : C::kColL + w * N) + c;
      uint32_t o[8];
      tmem_get<8>(at, o);
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f[k]);
      tmem_st8(at, o);
    }
  }
  tmem_wait_st();
}

// The work of the whole call as a list of units (every problem: kSegCost<N> for
// starting it, then its tiles), cut evenly: what this thread and this CTA have
// of it. Every thread takes a run of entries; what lies before it by a scan.
struct Plan {
  int e0, e1, before_u, before_p;  // the thread's entries; units and problems before them
  int u0, u1, per, extra;          // the CTA's units; units of every CTA, and how many CTAs have one more
};
template <int N, int kThreads>
__device__ __forceinline__ Plan plan_units(const Params& p, int* scan) {
  const int H = p.a.cache.H, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Plan plan;
  const int run = (p.E + kThreads - 1) / kThreads;
  plan.e0 = threadIdx.x * run, plan.e1 = min(p.E, plan.e0 + run);
  int units = 0, probs = 0;
  for (int e = plan.e0; e < plan.e1; ++e) {
    const int nt = entry_of<N>(p, e).nt;
    units += nt > 0 ? (nt + kSegCost<N>) * H : 0;
    probs += nt > 0 ? H : 0;
  }
  int iu = units, ip = probs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, iu, o), b = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) iu += a, ip += b;
  }
  if (lane == 31) scan[warp] = iu, scan[32 + warp] = ip;
  __syncthreads();
  int U = 0;
  plan.before_u = plan.before_p = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) plan.before_u += scan[w], plan.before_p += scan[32 + w];
    U += scan[w];
  }
  plan.before_u += iu - units;
  plan.before_p += ip - probs;
  // the first U % ctas CTAs take one unit more
  plan.per = U / static_cast<int>(gridDim.x), plan.extra = U - plan.per * static_cast<int>(gridDim.x);
  const int me = blockIdx.x;
  plan.u0 = me * plan.per + min(me, plan.extra), plan.u1 = plan.u0 + plan.per + (me < plan.extra ? 1 : 0);
  return plan;
}

// Segments seg0 .. seg0 + kSegs - 1 of the CTA into segs; returns how many it
// has in all. The whole block takes part.
template <int N>
__device__ __forceinline__ int plan_segments(const Params& p, const Plan& plan, int seg0, Seg* segs, int* first_seg,
                                             int* last_seg, int* has_tail) {
  const int H = p.a.cache.H;
  for (int pass = seg0 == 0 ? 0 : 1; pass < 2; ++pass) {
    // pass 0 finds the first and the last problem of this CTA (one that has only its start here is the next CTA's),
    // pass 1 writes the segments of this batch
    int u = plan.before_u, q = plan.before_p;
    for (int e = plan.e0; e < plan.e1 && plan.u0 < plan.u1; ++e) {
      const Entry en = entry_of<N>(p, e);
      // a problem's units: kSegCost<N> for starting it, then its tiles
      const int one = en.nt > 0 ? en.nt + kSegCost<N> : 0, all = one * H;
      if (en.nt > 0 && u < plan.u1 && u + all > plan.u0) {
        const int h0 = max(0, (plan.u0 - u) / one), h1 = min(H - 1, (plan.u1 - 1 - u) / one);
        for (int h = h0; h <= h1; ++h) {
          const int a = u + h * one + kSegCost<N>, z = a + en.nt;  // units of its tiles
          const int b0 = max(a, plan.u0), b1 = min(z, plan.u1);
          if (b1 <= b0) continue;
          if (pass == 0) {
            // (the CTA's other problems lie between these two, with tiles each)
            if (a - kSegCost<N> <= plan.u0) *first_seg = q + h;
            atomicMax(last_seg, q + h);
            continue;
          }
          const int i = q + h - *first_seg - seg0;
          if (i < 0 || i >= kSegs) continue;
          Seg s;
          s.b = en.b, s.h = h, s.rt = en.rt, s.j0 = b0 - a, s.nt = b1 - b0;
          s.row0 = en.row0, s.T = en.T, s.L = en.L;
          const bool starts = b0 == a, ends = b1 == z;
          s.slot = starts && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
          segs[i] = s;
          if (starts && !ends) {
            int* t = p.tails + 8 * blockIdx.x;
            t[0] = min(N, en.T * p.group - en.rt * N);
            // the CTA of the problem's last unit
            t[1] = z - 1 < plan.extra * (plan.per + 1) ? (z - 1) / (plan.per + 1) : plan.extra + (z - 1 - plan.extra * (plan.per + 1)) / plan.per;
            t[2] = en.row0;
            t[3] = en.rt;
            t[4] = h;
            *has_tail = 1;
          }
        }
      }
      u += all;
      q += en.nt > 0 ? H : 0;
    }
    __syncthreads();
  }
  return *last_seg - *first_seg + 1;
}

// A loading warp: the K tiles of the segments, or the V tiles with the scales of
// both, page by page into the ring. The scales go along as bytes, or (scales not
// null) through registers and into shared memory as floats, with the keys that are
// there as bits.
template <class C, class W>
__device__ __forceinline__ void load_tiles(const Params& p, uint8_t* smem, const Seg* segs, int count, int g, bool is_v,
                                           uint64_t* full, uint64_t* empty, uint32_t* good, volatile int* issued,
                                           W& wait, bool elected, int lane, float* scales = nullptr,
                                           uint32_t* lives = nullptr, uint64_t* c_full = nullptr,
                                           uint64_t* c_free = nullptr) {
  const int H = p.a.cache.H, ps = p.a.cache.page_size, ps_log = 31 - __clz(ps), ppt = 128 >> ps_log;
  // lane l < 16 copies bytes 16 l .. of a tile's 256 bytes of scales, which are those of page l * 8 / ps
  const int spage = (lane * 8 >> ps_log) & (ppt - 1), soff = (lane & 15) * 16 - (spage << (ps_log + 1));
  const uint32_t page_bytes = ps * C::kD, tile_pages = (1u << ppt) - 1u;
  const CUtensorMap* map = is_v ? &p.tm_v : &p.tm_k;
  uint8_t* ring = smem + (is_v ? C::kOffV : C::kOffK);
  int st = g % C::kStages;
  uint32_t par = (g / C::kStages - 1) & 1;
  for (int i = 0, gg = g; i < count; ++i) {
    const Seg s = segs[i];
    const int* table = p.a.page_table + s.b * p.a.page_table_stride;
    const int pages = (s.L + ps - 1) >> ps_log;
    // (page, head) of pages base .. base + 31, one a lane (-1: not there); those of the 32 after them in `next`
    int base = s.j0 * ppt;
    int next = base + lane < pages ? table[base + lane] : -1;
    int ids = 0;
    uint32_t valid = 0u;
    base -= 32;
    // Scales of tile t's keys 4 l .. 4 l + 3 for lane l, two tiles ahead of their use: their latency is that of memory.
    auto fetch = [&](int t, uint32_t& k, uint32_t& v) {
      const int x = t * ppt - base + (lane * 4 >> ps_log);
      const int here = __shfl_sync(0xffffffffu, ids, x & 31), then = __shfl_sync(0xffffffffu, next, x & 31);
      const bool ok = x < 32 ? valid >> (x & 31) & 1u
                             : x < 64 && static_cast<uint32_t>(then) < static_cast<uint32_t>(p.a.cache.num_pages);
      k = v = 0u;
      if (ok && t < s.j0 + s.nt) {
        const uint32_t ph = x < 32 ? here : then * H + s.h;
        const uint8_t* ex = p.a.cache.exps + (static_cast<size_t>(ph) << (ps_log + 1)) + (lane * 4 & (ps - 1));
        k = *reinterpret_cast<const uint32_t*>(ex);
        v = *reinterpret_cast<const uint32_t*>(ex + ps);
      }
    };
    uint32_t k0 = 0u, v0 = 0u, k1 = 0u, v1 = 0u;
    for (int j = s.j0; j < s.j0 + s.nt; ++j, ++gg) {
      if (j * ppt >= base + 32) {
        base += 32;
        const bool there = static_cast<uint32_t>(next) < static_cast<uint32_t>(p.a.cache.num_pages);
        ids = next * H + s.h;
        valid = __ballot_sync(0xffffffffu, there);
        next = base + 32 + lane < pages ? table[base + 32 + lane] : -1;
        if (is_v && scales && j == s.j0) {
          fetch(j, k0, v0);
          fetch(j + 1, k1, v1);
        }
      }
      const int at = j * ppt - base;
      const uint32_t have = valid >> at & tile_pages;
      uint32_t ek = 0u, ev = 0u;
      if (is_v && scales) {
        ek = k0, ev = v0, k0 = k1, v0 = v1;
        fetch(j + 2, k1, v1);
      }
      if (gg >= C::kStages) wait.warp(empty + st, par, is_v ? kErrVEmpty : kErrKEmpty);
      if (!wait.dead) {
        if (elected) {
          // before the arrival, which releases them to those who wait for the tile
          if (is_v && !scales) good[st] = have;
          issued[is_v] = gg + 1;
          mbar_arrive_expect_tx(full + st, __popc(have) * page_bytes);
        }
        uint32_t dst = smem_u32(ring + st * C::kTile);
        for (int x = 0; x < ppt; ++x, dst += page_bytes) {
          const int ph = __shfl_sync(0xffffffffu, ids, at + x);
          if (elected && (have >> x & 1u)) tma_load(dst, map, full + st, ph);
        }
        if (is_v && !scales) {
          const int ph = __shfl_sync(0xffffffffu, ids, at + spage);
          if (lane < 16) {
            if (have >> spage & 1u)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem + C::kOffE + st * 256 + lane * 16)),
                           "l"(p.a.cache.exps + (static_cast<size_t>(static_cast<uint32_t>(ph)) << (ps_log + 1)) + soff)
                           : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full + st)) : "memory");
          }
        }
      }
      if (is_v && scales) {
        constexpr int kScl = 4;
        const int sc = gg % kScl;
        if (gg >= kScl) wait.warp(c_free + sc, (gg / kScl - 1) & 1, kErrScales);
        const uint32_t there = have >> (lane * 4 >> ps_log) & 1u;
        uint32_t bits = 0u;
        float k2[4], v1[4], v2[4];  // 2^ek, ev and 2^-ev; byte 255 is NaN, byte 0 (never written) taken as the next
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t k = ek >> 8 * x & 255u, v = ev >> 8 * x & 255u;
          k2[x] = k == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(max(k, 1u) << 23);
          v1[x] = v == 255u ? __uint_as_float(0x7FC00000u) : static_cast<float>(v) - 127.f;
          v2[x] = __uint_as_float(min(max(254u - v, 1u), 254u) << 23);
          bits |= (there && 128 * j + 4 * lane + x < s.L ? 1u : 0u) << x;
        }
        float4* dst = reinterpret_cast<float4*>(scales + sc * 384) + lane;
        dst[0] = make_float4(k2[0], k2[1], k2[2], k2[3]);
        dst[32] = make_float4(v1[0], v1[1], v1[2], v1[3]);
        dst[64] = make_float4(v2[0], v2[1], v2[2], v2[3]);
        // the bits of eight lanes make a word
        bits <<= 4 * (lane & 7);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
        if ((lane & 7) == 0) lives[sc * 4 + (lane >> 3)] = bits;
        warp_arrive(c_full + sc);
      }
      if (++st == C::kStages) st = 0, par ^= 1u;
    }
  }
}

// The end of a CTA: its products and loads are over before its memory is given back.
template <int kStages>
__device__ __forceinline__ void finish(const Params& p, int warp, bool elected, uint64_t* drain, volatile int* abort_flag,
                                       const int* has_tail, volatile int* issued, volatile int* consumed, uint64_t* k_full,
                                       uint64_t* v_full) {
  // Drain: every issued MMA completes before tensor memory is released.
  if ((warp == 1 || warp == 2) && elected) {  // the thread that issued them
    uint64_t* d = drain + (warp - 1);
    mma_commit(d);
    bool done = false;
    const unsigned long long t0 = globaltimer_ns();
    while (!(done = mbar_try_wait(smem_u32(d), 0)) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
    }
    if (!done) atomicCAS(&g_cache_attn_error, 0, kErrDrain);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (!*has_tail) p.tails[8 * blockIdx.x] = 0;
    if (*abort_flag) {
      // bounded drain of loads that were issued but never consumed
      for (int x = 0; x < 2; ++x) {
        uint64_t* full = x ? v_full : k_full;
        for (int t = max(consumed[x], issued[x] - kStages); t < issued[x]; ++t) {  // (a stage loaded again was waited for)
          const unsigned long long t0 = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(full + t % kStages), (t / kStages) & 1) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
          }
        }
      }
    }
  }
  __syncthreads();
}

// A wait that fails raises the abort flag; every role then runs its loops to
// their end with waits that return at once, so the barriers of the softmax
// warps and of the block are always reached by all their threads.
template <int D, int N>
__global__ void __launch_bounds__(Cfg<D, N>::kThreads, 1) cache_attn_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, N>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Seg* segs = reinterpret_cast<Seg*>(smem + C::kOffSeg);
  float* qmul = reinterpret_cast<float*>(smem + C::kOffF);  // [2][N]
  float* nbias = reinterpret_cast<float*>(smem + C::kOffBias);  // [2][kPar][N]: kPLog2 - reference maximum
  float* lsum = reinterpret_cast<float*>(smem + C::kOffMax) + 4 * C::kPar * N;  // [2][kPar][4][N], behind wmax [kPar][4][N]
  float* fin = lsum + 8 * C::kPar * N;                      // [kPar + 1][N]: weights of the parities, 1 / l
  int* lim = reinterpret_cast<int*>(smem + C::kOffAlpha) + C::kPar * N;  // [2][N]: last key a row sees (without a tree)
  uint32_t* win = reinterpret_cast<uint32_t*>(smem + C::kOffWin);        // [kPar][4][N]: which of a tile's keys a row sees
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_full = bars;                // [stage]
  uint64_t* v_full = k_full + kStages;    // [stage]
  uint64_t* k_empty = v_full + kStages;   // [stage]: read by S
  uint64_t* v_empty = k_empty + kStages;  // [stage]: read by PV
  uint64_t* s_full = v_empty + kStages;  // [tile parity]
  uint64_t* s_free = s_full + C::kPar;    // [parity], 4 kHalves arrivals
  uint64_t* p_full = s_free + C::kPar;    // [parity], 4 kHalves arrivals
  uint64_t* o_done = p_full + C::kPar;          // [parity]: PV of the tile completed
  uint64_t* q_full = o_done + C::kPar;          // [buffer], 16 arrivals: the query rows' terms are there
  uint64_t* epi = q_full + 2;              // 16 arrivals: O of a segment was read
  uint64_t* drain = epi + 1;              // [2]
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* issued = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);     // [2]: tiles of K, of V loaded
  volatile int* consumed = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);  // [2]: and read
  int* first_seg = reinterpret_cast<int*>(smem + C::kOffMisc + 24);
  int* last_seg = reinterpret_cast<int*>(smem + C::kOffMisc + 28);
  int* has_tail = reinterpret_cast<int*>(smem + C::kOffMisc + 32);
  int* scan = reinterpret_cast<int*>(smem + C::kOffScan);  // [2][32]
  uint32_t* good = reinterpret_cast<uint32_t*>(scan + 64);  // [stage]: pages of the tile that are there

  // (uniform for the compiler, as is the elected thread: a tensor-core instruction issued under a thread's own branch
  // costs 53 cycles, under these 23 to 48)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool elected = elect_one();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(v_full + s, 1 + 16);  // the codes' loads, 16 lanes' copies of scales
      mbar_init(k_empty + s, 1);
      mbar_init(v_empty + s, 1);
    }
    for (int w = 0; w < C::kPar; ++w) {
      mbar_init(s_full + w, 1);
      mbar_init(s_free + w, 4 * C::kHalves);
      mbar_init(p_full + w, 4 * C::kHalves);
      mbar_init(o_done + w, 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(q_full + w, 16);
      mbar_init(drain + w, 1);
    }
    mbar_init(epi, 16);
    *abort_flag = 0;
    issued[0] = issued[1] = consumed[0] = consumed[1] = 0;
    *has_tail = 0;
    *first_seg = 0;
    *last_seg = -1;
    fence_barrier_init();
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), C::kCols);
    tmem_relinquish();
  }
  // nothing above touches global memory; the stream predecessor's results are read from here on
  griddep_wait();

  tc_fence_before();
  const Plan plan = plan_units<N, C::kThreads>(p, scan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Waiter<true> wait{abort_flag};
  int seg0 = 0, nsegs = 0;
  int g = 0;  // tiles so far; every role counts the same ones
  // Segments are planned kSegs at a time (one pass unless the sequences are many and short).
  do {
    __syncthreads();
    nsegs = plan_segments<N>(p, plan, seg0, segs, first_seg, last_seg, has_tail);
    const int count = min(kSegs, nsegs - seg0);

    if (warp == 0 || warp == 3) {
      load_tiles<C>(p, smem, segs, count, g, warp != 0, warp != 0 ? v_full : k_full, warp != 0 ? v_empty : k_empty, good,
                    issued, wait, elected, lane);
    } else if (warp == 1) {
      // ---------------------------------------------------------- PV issuer
      constexpr uint32_t kPV = idesc(D, 3 * N, 1, 1, 1);
      for (int i = 0, gg = g; i < count; ++i) {
        const int nt = segs[i].nt, sg = seg0 + i;
        if (sg > 0) wait.warp(epi, (sg - 1) & 1, kErrEpi);
        for (int j = 0; j < nt; ++j, ++gg) {
          const int st = gg % kStages, w = gg % C::kPar;
          bool ok = wait.warp(p_full + w, (gg / C::kPar) & 1, kErrPFull);
          ok = wait.warp(v_full + st, (gg / kStages) & 1, kErrVFull) && ok;
          if (!ok) continue;
          tc_fence_after();
          const uint64_t v = make_smem_desc(smem_u32(smem + C::kOffV + st * C::kTile), 16, 8 * D, swz_of(D));
          const uint64_t pd =
              make_smem_desc(smem_u32(smem + C::kOffP + w * C::kPTile), 16, 8 * C::kPP, swz_of(C::kPP));
          const uint32_t o = tmem + C::kColO + w * 3 * N;
          if (elected) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8f6f4_ss(o, v + ((kk * 32 * D) >> 4), pd + ((kk * 32 * C::kPP) >> 4), kPV,
                            (j >= C::kPar || kk > 0) ? 1u : 0u);
            mma_commit(v_empty + st);
            mma_commit(o_done + w);
            consumed[1] = gg + 1;
          }
          __syncwarp();
        }
      }
    } else if (warp == 2) {
      // ----------------------------------------------------------- S issuer
      constexpr uint32_t kS = idesc(128, N, 0, 0);
      for (int i = 0, gg = g; i < count; ++i) {
        const int nt = segs[i].nt, sg = seg0 + i;
        wait.warp(q_full + (sg & 1), (sg >> 1) & 1, kErrQFull);
        tc_fence_after();
        const uint8_t* qb = smem + C::kOffQ + (sg & 1) * 2 * C::kQ;
        const uint64_t q = make_smem_desc(smem_u32(qb), 16, 8 * D, swz_of(D));
        for (int j = 0; j < nt; ++j, ++gg) {
          const int st = gg % kStages, w = gg % C::kPar;
          bool ok = wait.warp(k_full + st, (gg / kStages) & 1, kErrKFull);
          if (gg >= C::kPar) ok = wait.warp(s_free + w, (gg / C::kPar - 1) & 1, kErrSFree) && ok;
          if (!ok) continue;
          tc_fence_after();
          const uint64_t k = make_smem_desc(smem_u32(smem + C::kOffK + st * C::kTile), 16, 8 * D, swz_of(D));
          const uint32_t s = tmem + C::kColS + w * N;
          if (elected) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_f8f6f4_ss(s, k + 2 * kk, q + (C::kQ >> 4) * t + 2 * kk, kS, t + kk > 0 ? 1u : 0u);
            mma_commit(s_full + w);
            mma_commit(k_empty + st);
            consumed[0] = gg + 1;
          }
          __syncwarp();
        }
      }
    } else {
      // ------------------------------------------------------------ softmax
      const int wg = (warp - 4) >> 2, w = wg % C::kPar, half = wg / C::kPar, q4 = warp & 3;
      const int lo_row = half * C::kHalf, hi_row = lo_row + C::kHalf;  // query rows of the warpgroup
      const int tid = q4 * 32 + lane;                      // key of a tile
      const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
      const uint32_t t_s = tmem + lane_off + C::kColS + w * N, t_l = tmem + lane_off + C::kColL + w * N;
      const uint32_t t_o = tmem + lane_off + C::kColO;
      const int ps = p.a.cache.page_size, ps_log = 31 - __clz(ps);
      uint8_t* p_tile = smem + C::kOffP + w * C::kPTile;
      const uint32_t* seen = win + (w * 4 + q4) * N;
      int gg = g;
      uint8_t* q_buf = smem + C::kOffQ;
      if (count > 0) load_rows<D, N, 16>(p, segs[0], q_buf + (seg0 & 1) * 2 * C::kQ, warp - 4, lane);
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        const Seg s = segs[i];
        const int sg = seg0 + i, buf = sg & 1;
        // A Q buffer is filled again two segments on: by then every tile of its segment has left the tensor core (this
        // warp has waited for them in the epilogue of the segment between).
        split_rows<D, N, 16>(p, s, q_buf + buf * 2 * C::kQ, qmul + buf * N, lim + buf * N, warp - 4, lane);
        warp_arrive(q_full + buf);
        if (i + 1 < count) load_rows<D, N, 16>(p, segs[i + 1], q_buf + (buf ^ 1) * 2 * C::kQ, warp - 4, lane);
        const int rows = min(hi_row, s.T * p.group - s.rt * N);  // this warpgroup's end where the tile's last row
        const int first = s.L - s.T;
        float* nb = nbias + (buf * C::kPar + w) * N;
        const float* qm = qmul + buf * N;
        // every row sees all keys up to this one
        const int least = p.a.tree ? first - 1 : (p.a.causal ? first + (s.rt * N) / p.group : s.L - 1);
        wait.warp(q_full + buf, (sg >> 1) & 1, kErrQFull);
        if (tid < C::kHalf) nb[lo_row + tid] = kPLog2 - kNever;
        {
          const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll 1
          for (int c = lo_row; c < rows; c += 8) tmem_st8(t_l + c, zero);
          tmem_wait_st();
        }
        named_sync(1 + wg, 128);
        const int g_end = gg + s.nt;
        int mine = 0;  // tiles of this warpgroup in the segment
        // its first tile, and the stage and phase of that, kept up without divisions
        const int skip = (w - gg) & (C::kPar - 1);
        int j = s.j0 + skip, it = (gg + skip) / C::kPar, st = (gg + skip) % kStages;
        uint32_t phase = ((gg + skip) / kStages) & 1;
        const int j_end = s.j0 + s.nt;
        gg = g_end;
#pragma unroll 1
        for (; j < j_end; j += C::kPar, ++it) {
          const int page = tid >> ps_log;
          wait.warp(v_full + st, phase, kErrVFull);
          const uint32_t pages = good[st];
          const uint8_t* ex = smem + C::kOffE + st * 256 + ((page << ps_log) * 2) + (tid & (ps - 1));
          const uint32_t ek = ex[0], ev = ex[ps];
          const bool live = 128 * j + tid < s.L && ((pages >> page) & 1u);
          const bool full = 128 * j + 128 <= s.L && pages == (1u << (128 >> ps_log)) - 1u;  // all keys are live
          // 2^ek and ev as floats; byte 255 is NaN, byte 0 (never written) taken as the next
          const float km = ek == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(max(ek, 1u) << 23);
          const float evf = ev == 255u ? __uint_as_float(0x7FC00000u) : static_cast<float>(ev) - 127.f;
          const float inv = __uint_as_float(min(max(254u - ev, 1u), 254u) << 23);  // 2^-ev
          const uint64_t km2 = f2_pack(km, km), ev2 = f2_pack(evf, evf), inv2 = f2_pack(inv, inv);
          const bool masked = !full || 128 * j + 127 > least;
          const uint32_t bit = live ? 1u << lane : 0u;
          if (masked) {
            // thread r works out which of the tile's keys row r sees
            if (tid < C::kHalf) {
              const int row = lo_row + tid, t = (s.rt * N + row) / p.group;
              const long long* words =
                  p.a.tree + (p.a.q_start ? static_cast<long long>(s.row0 + t) * p.a.tree_words
                                          : s.b * p.a.tree_sb + static_cast<long long>(t) * p.a.tree_words);
              const int last = lim[buf * N + row];
#pragma unroll 1
              for (int x = 0; x < 4; ++x) {
                const int k0 = 128 * j + 32 * x;
                uint32_t m;
                if (p.a.tree && row < rows) {
                  // drafted tokens k0 - first ..: their bits; the tokens before them are all seen
                  const int d0 = k0 - first, d1 = max(d0, 0), at = d1 >> 6, sh = d1 & 63;
                  unsigned long long lo = at < p.a.tree_words ? static_cast<unsigned long long>(words[at]) >> sh : 0ull;
                  if (sh > 32 && at + 1 < p.a.tree_words)
                    lo |= static_cast<unsigned long long>(words[at + 1]) << (64 - sh);
                  const int before = d1 - d0;
                  m = before >= 32 ? 0xFFFFFFFFu : (static_cast<uint32_t>(lo) << before) | ((1u << before) - 1u);
                } else {
                  const int n = last - k0 + 1;
                  m = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
                }
                win[(w * 4 + x) * N + row] = m;
              }
            }
            named_sync(1 + wg, 128);
          }
          wait.warp(s_full + w, it & 1, kErrSFull);
          tc_fence_after();
          if (lo_row >= rows) {  // none of its rows are there
            tc_fence_before();
            warp_arrive(s_free + w);
          }
          bool idle = it == 0;  // P and O of the warpgroup's previous tile are done with
#pragma unroll 1
          for (int c0 = lo_row; c0 < rows; c0 += C::kGroup) {
            constexpr int kG = C::kGroup;
            uint64_t x[kG / 2];  // two rows each: the exponent of P (score, reference maximum, V's scale), then P
#pragma unroll 1
            for (bool moved = false;; moved = true) {
              uint32_t r[kG];
              tmem_get<kG>(t_s + c0, r);
#pragma unroll
              for (int c = 0; c < kG; c += 4) {
                const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(qm + c0 + c);
                const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(nb + c0 + c);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint64_t acc = f2_pack(__uint_as_float(r[c + 2 * k]), __uint_as_float(r[c + 2 * k + 1]));
                  x[c / 2 + k] = f2_add(f2_fma(f2_mul(acc, k ? qv.y : qv.x), km2, k ? bv.y : bv.x), ev2);
                }
              }
              if (masked) {
#pragma unroll
                for (int c = 0; c < kG; c += 4) {
                  const uint4 m = *reinterpret_cast<const uint4*>(seen + c0 + c);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    float a, b;
                    f2_unpack(x[c / 2 + k], a, b);
                    x[c / 2 + k] = f2_pack(((k ? m.z : m.x) & bit) ? a : -INFINITY, ((k ? m.w : m.y) & bit) ? b : -INFINITY);
                  }
                }
              }
              if (moved) {
                // (the steps of scores of 2^27 and more can carry P past its largest even so)
#pragma unroll
                for (int c = 0; c < kG / 2; ++c) x[c] = at_most(x[c], kPTop);
                break;
              }
              float top = -INFINITY;
#pragma unroll
              for (int c = 0; c < kG / 2; ++c) {
                float a, b;
                f2_unpack(x[c], a, b);
                top = fmax3(top, a, b);
              }
              if (!named_any(1 + wg, 128, top > kPTop)) break;
              if (mine > 0) {
                if (!idle) wait.warp(o_done + w, (it - 1) & 1, kErrODone);
                idle = true;
              }
              move_references<D, N>(smem, tmem, c0, wg, buf, km, evf, bit, masked, mine > 0);
            }
            if (c0 + kG >= rows) {
              tc_fence_before();
              warp_arrive(s_free + w);
            }
            if (!idle) wait.warp(o_done + w, (it - 1) & 1, kErrODone);
            idle = true;
            uint32_t hi[kG / 4], mid[kG / 4], lo[kG / 4];
#pragma unroll
            for (int c = 0; c < kG; c += 4) {
              float q[4];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float a, b;
                f2_unpack(x[c / 2 + k], a, b);
                q[2 * k] = ex2_approx(a);
                q[2 * k + 1] = ex2_approx(b);
                x[c / 2 + k] = f2_pack(q[2 * k], q[2 * k + 1]);
              }
              split_p(q[0], q[1], q[2], q[3], hi[c / 4], mid[c / 4], lo[c / 4]);
            }
            const uint32_t at = tid * C::kPP + c0;
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              const uint32_t* t = z == 0 ? hi : (z == 1 ? mid : lo);
              uint8_t* dst = p_tile + swizzled<C::kPP>(at + z * N);
              if (kG == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(t[0], t[1]);
              else *reinterpret_cast<uint4*>(dst) = make_uint4(t[0], t[1], t[kG / 4 - 2], t[kG / 4 - 1]);
            }
            uint32_t l[kG];
            tmem_get<kG>(t_l + c0, l);
#pragma unroll
            for (int c = 0; c < kG; c += 2) {
              float a, b;
              f2_unpack(f2_fma(x[c / 2], inv2, f2_pack(__uint_as_float(l[c]), __uint_as_float(l[c + 1]))), a, b);
              l[c] = __float_as_uint(a);
              l[c + 1] = __float_as_uint(b);
            }
            tmem_put<kG>(t_l + c0, l);
          }
          // (a warpgroup without rows must not arrive for a tile whose predecessor the other half still works on)
          if (!idle) wait.warp(o_done + w, (it - 1) & 1, kErrODone);
          if (!full && lo_row == 0) {
            // what lies behind the sequence, or in a page that is not there, may be NaN: 0 * NaN would reach O
            if (!live) {
              uint4* row = reinterpret_cast<uint4*>(smem + C::kOffV + st * C::kTile + tid * D);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) row[k] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          tmem_wait_st();
          fence_proxy_async_shared();
          tc_fence_before();
          warp_arrive(p_full + w);
          ++mine;
          st += C::kPar;
          if (st >= kStages) st -= kStages, phase ^= 1u;
        }
        // ---------------------------------------------------------- epilogue
        // Row sums of the warp's 32 keys, eight rows at a time: each step
        // halves the rows a lane holds and doubles the keys they stand for.
        float* ls = lsum + ((buf * C::kPar + w) * 4 + q4) * N;
#pragma unroll 1
        for (int c = lo_row; c < rows; c += 8) {
          uint32_t a[8];
          tmem_ld8(t_l + c, a);
          tmem_wait8(a);
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(a[k]);
#pragma unroll
          for (int o = 16, n = 4; n > 0; o >>= 1, n >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < n) {
                const float other = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + n], o);
                v[k] = (up ? v[k + n] : v[k]) + other;
              }
          }
          float x = v[0];  // row (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          if ((lane & 3) == 0) ls[c + (lane >> 2)] = x;
        }
        // tiles 0 .. g_end - 1 were issued; tiles of parity x among the first n: (n + kPar - 1 - x) / kPar
        uint32_t had = 0;  // bit x: parity x has tiles in this segment
#pragma unroll
        for (int x = 0; x < C::kPar; ++x) {
          const int n = (g_end + C::kPar - 1 - x) / C::kPar;
          if (n > (g_end - s.nt + C::kPar - 1 - x) / C::kPar) {
            had |= 1u << x;
            wait.warp(o_done + x, (n - 1) & 1, kErrODone);
          }
        }
        named_sync(5 + half, 128 * C::kPar);
        const int id = lo_row + w * 128 + tid;
        if (id < rows) {
          float m = kNever, sum = 0.f;
#pragma unroll
          for (int x = 0; x < C::kPar; ++x)
            if (had >> x & 1u) m = fmaxf(m, kPLog2 - nbias[(buf * C::kPar + x) * N + id]);
#pragma unroll
          for (int x = 0; x < C::kPar; ++x) {
            if (!(had >> x & 1u)) continue;
            const float a = ex2_approx(kPLog2 - nbias[(buf * C::kPar + x) * N + id] - m);
            const float* z = lsum + (buf * C::kPar + x) * 4 * N + id;
            sum += a * (z[0] + z[N] + z[2 * N] + z[3 * N]);
            fin[x * N + id] = a;
          }
          fin[C::kPar * N + id] = s.slot >= 0 ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);
          if (s.slot >= 0) {
            p.part_ml[(static_cast<size_t>(s.slot) * 2) * N + id] = m;
            p.part_ml[(static_cast<size_t>(s.slot) * 2 + 1) * N + id] = sum;
          } else if (p.a.lse) {
            const int t = (s.rt * N + id) / p.group, hq = s.h * p.group + (s.rt * N + id) - t * p.group;
            p.a.lse[static_cast<size_t>(s.row0 + t) * p.a.Hq + hq] =
                sum == 0.f ? -INFINITY : (m - kPLog2 + log2f(sum)) * kLn2;
          }
        }
        named_sync(5 + half, 128 * C::kPar);
        tc_fence_after();
        // M = 64 (d = 64) leaves 16 rows in each quarter of the lanes
        const int channel = D == 128 ? tid : q4 * 16 + (lane & 15);
        const bool holds = D == 128 || lane < 16;
#pragma unroll 1
        for (int c0 = lo_row + w * 8; c0 < rows; c0 += 8 * C::kPar) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = 0.f;
#pragma unroll 1
          for (int x = 0; x < C::kPar; ++x) {
            if (!(had >> x & 1u)) continue;
            uint32_t hi[8], mid[8], lo[8];
            const uint32_t at = t_o + x * 3 * N + c0;
            tmem_ld8(at, hi);
            tmem_ld8(at + N, mid);
            tmem_ld8(at + 2 * N, lo);
            tmem_wait8(hi);
            tmem_wait8(mid);
            tmem_wait8(lo);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o[k] = fmaf(fin[x * N + c0 + k],
                          fmaf(__uint_as_float(lo[k]), 1.f / kLoScale,
                               fmaf(__uint_as_float(mid[k]), 1.f / kMidScale, __uint_as_float(hi[k]))),
                          o[k]);
          }
          int t = (s.rt * N + c0) / p.group, hg = s.rt * N + c0 - t * p.group;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (holds && c0 + k < rows) {
              const float y = o[k] * fin[C::kPar * N + c0 + k];
              if (s.slot >= 0)
                p.part_o[(static_cast<size_t>(s.slot) * N + c0 + k) * D + channel] = y;
              else
                static_cast<__nv_bfloat16*>(p.a.out)[(static_cast<size_t>(s.row0 + t) * p.a.Hq + s.h * p.group + hg) * D +
                                                     channel] = __float2bfloat16(y);
            }
            if (++hg == p.group) hg = 0, ++t;
          }
        }
        tc_fence_before();
        warp_arrive(epi);
      }
    }
    // the tiles of this batch, for every role's next one
    for (int i = 0; i < count; ++i) g += segs[i].nt;
    seg0 += kSegs;
  } while (seg0 < nsegs);

  finish<kStages>(p, warp, elected, drain, abort_flag, has_tail, issued, consumed, k_full, v_full);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// Many query rows a KV head (drafted trees, chunks of prompts): a tile is 128
// query rows by 128 keys, S = Q K^T and O = P V with the rows on the tensor
// core's 128 rows, so that a row's maximum and sum stay with one thread a half of
// the keys and nothing is agreed on between warps. The softmax bounds it: 16384
// exponentials a tile are 1024 cycles of the special-function units and the
// products 1024 of the tensor core (d = 128), and two softmax warps a scheduler do not
// cover their latencies: a tile takes 3700 cycles, at 0.40 instructions a cycle and
// scheduler. A tree of 61 tokens, group 4, on 8 sequences of up to 16384: 158 us (164
// behind a pass that leaves L2 full of written lines), 0.30 of the measured bf16 rate; 3
// chunks of up to 1024 queries at up to 16384 tokens, d = 64: 448 us, d = 128: 492 us.
// Measured against it on the chunks (d = 64; P was two 8-bit terms then): 16 warps with
// two threads a row 531 us against 503; one S, P beside it 510; each half of the keys with
// its own S products 522; the exponentials of 32 keys beside the scores of the next 32 709.
//   Q in two E4M3 terms as above, K as it is; the scales of keys are
//   per column here: a loading warp writes 2^ek, ev and 2^-ev of a tile's keys to
//   shared memory
//   P in fp16 in tensor memory, and V as fp16 copies of its codes, which are exact, in
//   shared memory: P 2^ev is 2^10 or more for the row's largest, 11 bits down to 2^-24 of
//   that, an error of at most 2^-35 of it below. (In three E5M2 terms as above the splitting
//   would be twice the softmax's conversions.) Four warps make the copies: made by the softmax
//   warps, chunks and tree took 500, 544 and 172 us
// CTA (persistent, 512 threads): warps 0, 3 load, 1 issues P V, 2 issues Q K^T, 12-15 widen V,
// 4-11 softmax: warp 4 + 4 h + q has rows 32 q .. + 31 and keys 64 h .. + 63 of every
// tile, a thread a row, with its own reference maxima, sums and O, so that no lane
// waits on another and all lanes of a warp read the same scales; the halves are
// joined at a segment's end.
// Tensor memory: S [2][128], O [2 key halves][D]; P takes the place of the scores it
// was made of, so S of tile g + 2 follows P V of tile g.
// ---------------------------------------------------------------------------
template <int D>
struct Wide {
  static constexpr int kD = D, kThreads = 512, N = 128;
  // Registers a thread, 128 at launch: four warps that load and issue, four that widen V, eight of softmax. The chunks at
  // d = 128 take 491 us so, 518 with 88, 56 and 184, 540 with 112, 48 and 176, 511 with 104, 72 and 168.
  static constexpr int kRegsHelp = 96, kRegsWiden = 64, kRegsSoftmax = 176;
  static_assert(kRegsHelp + kRegsWiden + 2 * kRegsSoftmax <= 4 * 128, "registers");
  static constexpr int kTile = 128 * D, kQ = 128 * D;
  static constexpr int kScl = 4;                         // tiles of scales in flight
  static constexpr int kWords = kScl * (3 * 128 + 4) + 2 * 128 + 2 * 128 + 2 * 2 * 128;  // see the kernel
  static constexpr int kWide = 2 * kTile;                // bytes of a V tile in fp16
  static constexpr int kFixed = 4 * kQ + 2 * kWide + 4 * kWords + kSegs * static_cast<int>(sizeof(Seg)) + 1024;
  static constexpr int kRoom = (227 * 1024 - 1024 - kFixed) / (2 * kTile);
  static constexpr int kStages = kRoom > 8 ? 8 : kRoom;
  static constexpr int kOffK = 0, kOffV = kOffK + kStages * kTile;
  static constexpr int kOffQ = kOffV + kStages * kTile;  // [2 buffers][2 terms][128][D]
  static constexpr int kOffW = kOffQ + 4 * kQ;           // [2]: V in fp16
  static constexpr int kOffSeg = kOffW + 2 * kWide;
  static constexpr int kOffF = kOffSeg + kSegs * static_cast<int>(sizeof(Seg));
  static constexpr int kOffBar = (kOffF + 4 * kWords + 7) & ~7;
  static constexpr int kBars = 4 * kStages + 2 * 3 + 2 + 1 + 2 + 2 * kScl;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kOffScan = kOffMisc + 64;
  static constexpr int kBytes = kOffScan + 2 * 32 * 4;
  static constexpr int kSmem = kBytes + 1024;
  static_assert(kSmem <= 227 * 1024 && kStages >= 2 && kOffF % 16 == 0, "shared memory");
  static constexpr int kOffE = 0;                        // (no ring of scale bytes)
  static constexpr int kColS = 0, kColO = 256;           // S [2][128], O [2 key halves][D at 128 each]
};

// Drafted tokens first + d .. first + d + 31 of a tree's row as bits (d < 0: the tokens before them, all seen).
__device__ __forceinline__ uint32_t tree_bits(const long long* words, int n_words, int d) {
  const int d1 = max(d, 0), at = d1 >> 6, sh = d1 & 63, before = d1 - d;
  if (before >= 32) return 0xFFFFFFFFu;
  unsigned long long x = at < n_words ? static_cast<unsigned long long>(words[at]) >> sh : 0ull;
  if (sh > 32 && at + 1 < n_words) x |= static_cast<unsigned long long>(words[at + 1]) << (64 - sh);
  return (static_cast<uint32_t>(x) << before) | ((1u << before) - 1u);
}

template <int D>
__global__ void __launch_bounds__(Wide<D>::kThreads, 1) cache_attn_wide_kernel(const __grid_constant__ Params p) {
  using C = Wide<D>;
  constexpr int kStages = C::kStages, N = C::N;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Seg* segs = reinterpret_cast<Seg*>(smem + C::kOffSeg);
  float* scales = reinterpret_cast<float*>(smem + C::kOffF);          // [kScl][2^ek, ev, 2^-ev][128]
  uint32_t* lives = reinterpret_cast<uint32_t*>(scales + C::kScl * 384);  // [kScl][4]: keys that are there
  float* qmul = reinterpret_cast<float*>(lives + C::kScl * 4);        // [2][128]
  int* lim = reinterpret_cast<int*>(qmul + 2 * N);                    // [2][128]
  float* fin = reinterpret_cast<float*>(lim + 2 * N);                 // [2 key halves][reference, l][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_full = bars;                // [stage]
  uint64_t* v_full = k_full + kStages;    // [stage]
  uint64_t* k_empty = v_full + kStages;   // [stage]
  uint64_t* v_empty = k_empty + kStages;  // [stage]: widened to fp16
  uint64_t* s_full = v_empty + kStages;   // [tile parity]: scores and scales, 2 arrivals
  uint64_t* p_full = s_full + 2;          // [tile parity], 8 arrivals
  uint64_t* o_done = p_full + 2;          // [tile parity]
  uint64_t* q_full = o_done + 2;          // [buffer], 8 arrivals
  uint64_t* epi = q_full + 2;             // 8 arrivals
  uint64_t* drain = epi + 1;              // [2]
  uint64_t* c_full = drain + 2;           // [kScl]: a tile's scales are written
  uint64_t* c_free = c_full + C::kScl;    // [kScl], 9 arrivals: and were read
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* issued = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  volatile int* consumed = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);
  int* first_seg = reinterpret_cast<int*>(smem + C::kOffMisc + 24);
  int* last_seg = reinterpret_cast<int*>(smem + C::kOffMisc + 28);
  int* has_tail = reinterpret_cast<int*>(smem + C::kOffMisc + 32);
  int* scan = reinterpret_cast<int*>(smem + C::kOffScan);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool elected = elect_one();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(k_empty + s, 1);
      mbar_init(v_empty + s, 4);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(s_full + w, 2);
      mbar_init(p_full + w, 12);
      mbar_init(o_done + w, 1);
      mbar_init(q_full + w, 8);
      mbar_init(drain + w, 1);
    }
    mbar_init(epi, 8);
    for (int s = 0; s < C::kScl; ++s) mbar_init(c_full + s, 1), mbar_init(c_free + s, 12);
    *abort_flag = 0;
    issued[0] = issued[1] = consumed[0] = consumed[1] = 0;
    *has_tail = 0;
    *first_seg = 0;
    *last_seg = -1;
    fence_barrier_init();
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(const_cast<uint32_t*>(tmem_slot), 512);
    tmem_relinquish();
  }
  griddep_wait();
  tc_fence_before();
  const Plan plan = plan_units<N, C::kThreads>(p, scan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Waiter<false> wait{abort_flag};
  int seg0 = 0, nsegs = 0;
  int g = 0;
  // The next batch of segments; every role plans with the block and then counts the same tiles.
  auto next = [&]() {
    __syncthreads();
    nsegs = plan_segments<N>(p, plan, seg0, segs, first_seg, last_seg, has_tail);
    return min(kSegs, nsegs - seg0);
  };
  auto more = [&](int count) {
    for (int i = 0; i < count; ++i) g += segs[i].nt;
    seg0 += kSegs;
    return seg0 < nsegs;
  };
  if (warp < 4) {
    reg_dealloc<C::kRegsHelp>();
    int count;
    do {
      count = next();
      if (warp == 0 || warp == 3) {
        load_tiles<C>(p, smem, segs, count, g, warp != 0, warp != 0 ? v_full : k_full, warp != 0 ? v_empty : k_empty,
                      nullptr, issued, wait, elected, lane, scales, lives, c_full, c_free);
      } else if (warp == 1) {
        // ---------------------------------------------------------- PV issuer
        constexpr uint32_t kPV = idesc(128, D, 0, 1);
        for (int i = 0, gg = g; i < count; ++i) {
          const int nt = segs[i].nt, sg = seg0 + i;
          for (int j = 0; j < nt; ++j, ++gg) {
            const int w = gg & 1;
            if (j == 0 && sg > 0) wait.warp(epi, (sg - 1) & 1, kErrEpi);
            if (!wait.warp(p_full + w, (gg >> 1) & 1, kErrPFull)) continue;
            tc_fence_after();
            // 64 channels of a key are 128 bytes; the next 64 lie a whole tile of keys on
            const uint64_t v = make_smem_desc(smem_u32(smem + C::kOffW + w * C::kWide), 128 * 128, 8 * 128, swz_of(128));
            const uint32_t pt = tmem + C::kColS + w * 128;
            if (elected) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_f16_ts(tmem + C::kColO + h * 128, pt + h * 64 + 8 * kk, v + (((4 * h + kk) * 16 * 128) >> 4), kPV,
                             (j > 0 || kk > 0) ? 1u : 0u);
              mma_commit(o_done + w);
              consumed[1] = gg + 1;
            }
            __syncwarp();
          }
        }
      } else {
        // ----------------------------------------------------------- S issuer
        constexpr uint32_t kS = idesc(128, 128, 0, 0);
        for (int i = 0, gg = g; i < count; ++i) {
          const int nt = segs[i].nt, sg = seg0 + i;
          wait.warp(q_full + (sg & 1), (sg >> 1) & 1, kErrQFull);
          tc_fence_after();
          const uint64_t q = make_smem_desc(smem_u32(smem + C::kOffQ + (sg & 1) * 2 * C::kQ), 16, 8 * D, swz_of(D));
          for (int j = 0; j < nt; ++j, ++gg) {
            const int st = gg % kStages, w = gg & 1;
            bool ok = wait.warp(k_full + st, (gg / kStages) & 1, kErrKFull);
            if (gg >= 2) ok = wait.warp(o_done + w, ((gg >> 1) - 1) & 1, kErrODone) && ok;  // P lay in this S
            ok = wait.warp(c_full + gg % C::kScl, (gg / C::kScl) & 1, kErrScales) && ok;    // so that one wait does for both
            if (!ok) continue;
            tc_fence_after();
            const uint64_t k = make_smem_desc(smem_u32(smem + C::kOffK + st * C::kTile), 16, 8 * D, swz_of(D));
            const uint32_t s = tmem + C::kColS + w * 128;
            if (elected) {
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_f8f6f4_ss(s, q + (C::kQ >> 4) * t + 2 * kk, k + 2 * kk, kS, t + kk > 0 ? 1u : 0u);
              mma_commit(s_full + w);
              mbar_arrive(s_full + w);
              mma_commit(k_empty + st);
              consumed[0] = gg + 1;
            }
            __syncwarp();
          }
        }
      }
    } while (more(count));
  } else if (warp >= 12) {
    // --------------------------------------------------------------- V to fp16
    reg_dealloc<C::kRegsWiden>();
    const int key = threadIdx.x & 127;
    int count;
    do {
      count = next();
      int tiles = 0;
      for (int i = 0; i < count; ++i) tiles += segs[i].nt;
      for (int gg = g; gg < g + tiles; ++gg) {
        const int st = gg % kStages, sc = gg % C::kScl, w = gg & 1;
        wait.warp(v_full + st, (gg / kStages) & 1, kErrVFull);
        wait.warp(c_full + sc, (gg / C::kScl) & 1, kErrScales);
        if (gg >= 2) wait.warp(o_done + w, ((gg >> 1) - 1) & 1, kErrODone);  // the copy's last product
        widen_row<D, D / 16>(smem + C::kOffV + st * C::kTile, smem + C::kOffW + w * C::kWide, key, 0,
                             lives[sc * 4 + (key >> 5)] >> lane & 1u);
        fence_proxy_async_shared();
        warp_arrive(v_empty + st);
        warp_arrive(c_free + sc);
        warp_arrive(p_full + w);
      }
    } while (more(count));
  } else {
    reg_alloc<C::kRegsSoftmax>();
    int count;
    do {
      count = next();
      // ------------------------------------------------------------ softmax
      const int h = (warp - 4) >> 2, q4 = warp & 3;
      const int row = q4 * 32 + lane;  // of the tile
      const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
      uint8_t* q_buf = smem + C::kOffQ;
      int gg = g;
      if (count > 0) load_rows<D, N, 8>(p, segs[0], q_buf + (seg0 & 1) * 2 * C::kQ, warp - 4, lane);
#pragma unroll 1
      for (int i = 0; i < count; ++i) {
        const Seg s = segs[i];
        const int sg = seg0 + i, buf = sg & 1;
        split_rows<D, N, 8>(p, s, q_buf + buf * 2 * C::kQ, qmul + buf * N, lim + buf * N, warp - 4, lane);
        warp_arrive(q_full + buf);
        // (the other buffer's segment has left the tensor core: this warp saw its last tile done in the epilogue)
        if (i + 1 < count) load_rows<D, N, 8>(p, segs[i + 1], q_buf + (buf ^ 1) * 2 * C::kQ, warp - 4, lane);
        const int rows = min(N, s.T * p.group - s.rt * N), first = s.L - s.T;
        const int least = p.a.tree ? first - 1 : (p.a.causal ? first + (s.rt * N) / p.group : s.L - 1);
        wait.warp(q_full + buf, (sg >> 1) & 1, kErrQFull);
        const float qm = qmul[buf * N + row];
        const int last = lim[buf * N + row];
        const long long* words = nullptr;
        if (p.a.tree && row < rows) {
          const int t = (s.rt * N + row) / p.group;
          words = p.a.tree + (p.a.q_start ? static_cast<long long>(s.row0 + t) * p.a.tree_words
                                          : s.b * p.a.tree_sb + static_cast<long long>(t) * p.a.tree_words);
        }
        float nb = 0.f;      // kPLog2 - reference maximum of the row, 0 while no key was seen
        bool fresh = true;   // no key was seen
        uint64_t sum[2] = {0ull, 0ull};
        const int g_end = gg + s.nt;
#pragma unroll 1
        for (int j = s.j0; gg < g_end; ++gg, ++j) {
          const int sb = gg & 1;
          const int sc = gg % C::kScl;
          wait.warp(s_full + sb, (gg >> 1) & 1, kErrSFull);
          tc_fence_after();
          const ulonglong2* km = reinterpret_cast<const ulonglong2*>(scales + sc * 384 + 64 * h);
          const ulonglong2* ev = km + 32;
          const ulonglong2* iv = km + 64;
          const uint4 lv = *reinterpret_cast<const uint4*>(lives + sc * 4);
          uint64_t x[32];
          const uint64_t qm2 = f2_pack(qm, qm), nb2 = f2_pack(nb, nb);
          const uint32_t t_s = tmem + lane_off + C::kColS + sb * 128 + 64 * h;
          {
            uint32_t r[2][32];
            tmem_ld32(t_s, r[0]);
            tmem_ld32(t_s + 32, r[1]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              tmem_wait_ld(r[y]);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const ulonglong2 a = km[8 * y + k], b = ev[8 * y + k];
                const uint64_t r0 = f2_pack(__uint_as_float(r[y][4 * k]), __uint_as_float(r[y][4 * k + 1]));
                const uint64_t r1 = f2_pack(__uint_as_float(r[y][4 * k + 2]), __uint_as_float(r[y][4 * k + 3]));
                x[16 * y + 2 * k] = f2_add(f2_fma(f2_mul(r0, qm2), a.x, b.x), nb2);
                x[16 * y + 2 * k + 1] = f2_add(f2_fma(f2_mul(r1, qm2), a.y, b.y), nb2);
              }
            }
          }
          const bool full = (lv.x & lv.y & lv.z & lv.w) == ~0u;
          if (!full || 128 * j + 127 > least) {
            const uint32_t live[2] = {h ? lv.z : lv.x, h ? lv.w : lv.y};
            uint32_t see[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int k0 = 128 * j + 64 * h + 32 * k, n = last - k0 + 1;
              uint32_t m = n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
              if (words) m = tree_bits(words, p.a.tree_words, k0 - first);
              see[k] = m & live[k];
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float a, b;
              f2_unpack(x[k], a, b);
              const uint32_t m = see[k >> 4] >> ((2 * k) & 31);
              x[k] = f2_pack((m & 1u) ? a : -INFINITY, (m & 2u) ? b : -INFINITY);
            }
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float a, b;
            f2_unpack(x[k], a, b);
            tops[k & 3] = fmax3(tops[k & 3], a, b);
          }
          const float top = fmaxf(fmax3(tops[0], tops[1], tops[2]), tops[3]);
          if (__any_sync(0xffffffffu, top > kPTop || (fresh && top > -INFINITY))) {
            // some row's score passed its reference, or is its first: see move_references
            const bool moves = top > kPTop || (fresh && top > -INFINITY);
            const float now = moves ? reference(top, nb) : nb;
            const float factor = moves && !fresh ? ex2_approx(now - nb) : 1.f;
            const uint64_t d2 = f2_pack(now - nb, now - nb), f2 = f2_pack(factor, factor);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = f2_add(x[k], d2);
            sum[0] = f2_mul(sum[0], f2), sum[1] = f2_mul(sum[1], f2);
            nb = now;
            fresh = fresh && !moves;
            if (j > s.j0 && __any_sync(0xffffffffu, factor != 1.f)) {
              wait.warp(o_done + ((gg - 1) & 1), ((gg - 1) >> 1) & 1, kErrODone);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                const uint32_t at = tmem + lane_off + C::kColO + h * 128 + c;
                tmem_ld32(at, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * factor);
                tmem_st32(at, o);
              }
              tmem_wait_st();
            }
          }
          // over the scores that this warp has read
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const ulonglong2 c = iv[8 * y + k];
              float a0, a1, a2, a3;
              f2_unpack(x[16 * y + 2 * k], a0, a1);
              f2_unpack(x[16 * y + 2 * k + 1], a2, a3);
              a0 = ex2_approx(a0), a1 = ex2_approx(a1), a2 = ex2_approx(a2), a3 = ex2_approx(a3);
              sum[0] = f2_fma(f2_pack(a0, a1), c.x, sum[0]);
              sum[1] = f2_fma(f2_pack(a2, a3), c.y, sum[1]);
              w[2 * k] = half_p(a0, a1), w[2 * k + 1] = half_p(a2, a3);
            }
            tmem_st16(t_s + 16 * y, w);
          }
          warp_arrive(c_free + sc);
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(p_full + sb);
        }
        // ---------------------------------------------------------- epilogue
        float l0, l1;
        f2_unpack(f2_add(sum[0], sum[1]), l0, l1);
        l0 += l1;
        wait.warp(o_done + ((g_end - 1) & 1), ((g_end - 1) >> 1) & 1, kErrODone);
        fin[2 * h * N + row] = fresh ? kNever : kPLog2 - nb;
        fin[(2 * h + 1) * N + row] = l0;
        named_sync(1, 256);
        tc_fence_after();
        // half of the row's channels; the two key halves joined
        const float m0 = fin[row], m1 = fin[2 * N + row], m = fmaxf(m0, m1);
        float a0 = ex2_approx(m0 - m), a1 = ex2_approx(m1 - m);
        const float l = a0 * fin[N + row] + a1 * fin[3 * N + row];
        const int t = (s.rt * N + row) / p.group, hq = s.h * p.group + (s.rt * N + row) - t * p.group;
        if (h == 0 && row < rows) {
          if (s.slot >= 0) {
            p.part_ml[(static_cast<size_t>(s.slot) * 2) * N + row] = m;
            p.part_ml[(static_cast<size_t>(s.slot) * 2 + 1) * N + row] = l;
          } else if (p.a.lse) {
            p.a.lse[static_cast<size_t>(s.row0 + t) * p.a.Hq + hq] = l == 0.f ? -INFINITY : (m - kPLog2 + log2f(l)) * kLn2;
          }
        }
        if (s.slot < 0) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          a0 *= inv, a1 *= inv;
        }
#pragma unroll 1
        for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 16) {
          uint32_t o[16], o1[16];
          const uint32_t at = tmem + lane_off + C::kColO + c;
          tmem_get<16>(at, o);
          tmem_get<16>(at + 128, o1);
          float y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = fmaf(a0, __uint_as_float(o[k]), a1 * __uint_as_float(o1[k]));
          if (row < rows) {
            if (s.slot >= 0) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + static_cast<size_t>(s.slot) * N * D + c * N) + row;
#pragma unroll
              for (int k = 0; k < 4; ++k) dst[k * N] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            } else {
              uint32_t b[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const __nv_bfloat162 z = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
                b[k] = *reinterpret_cast<const uint32_t*>(&z);
              }
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) +
                                                    (static_cast<size_t>(s.row0 + t) * p.a.Hq + hq) * D + c);
              dst[0] = make_uint4(b[0], b[1], b[2], b[3]);
              dst[1] = make_uint4(b[4], b[5], b[6], b[7]);
            }
          }
        }
        tc_fence_before();
        warp_arrive(epi);
      }
    } while (more(count));
  }

  finish<kStages>(p, warp, elected, drain, abort_flag, has_tail, issued, consumed, k_full, v_full);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  griddep_launch_dependents();
}

// Joins the partial results of the problems that CTA boundaries cut: block x
// takes the one whose first piece is the last segment of CTA x, block y its
// query rows y * kRows .. . A row's warp w of kW takes pieces 4 w .. 4 w + 3 of every
// 4 kW, so that a row's loads are in flight at once; the warps' sums are added in
// order. Eight warps a row where few rows share many pieces; two of 128 rows, which
// have few (a row a block was 18944 blocks and 30 us there).
template <int N>
constexpr int kJoinRows = N == 128 ? 4 : 1;
template <int D, int N>
__global__ void __launch_bounds__(256) cache_attn_join_kernel(const __grid_constant__ Params p) {
  constexpr int kRows = kJoinRows<N>, kW = 8 / kRows;
  __shared__ float sm[8], sl[8], so[8][D];
  griddep_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y * kRows + warp / kW, sub = warp % kW;
  const int* tail = p.tails + 8 * c0;
  if (blockIdx.y * kRows < tail[0]) {
    const int pieces = r < tail[0] ? tail[1] - c0 + 1 : 0;
    constexpr int kPer = D / 32, kStep = 4;
    float m = kNever, sum = 0.f, acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int k0 = sub * kStep; k0 < pieces; k0 += kW * kStep) {
      float pm[kStep], pl[kStep], v[kStep][kPer];
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        // one piece past the last is read as a copy of it that counts nothing
        const int piece = min(k0 + k, pieces - 1);
        const size_t slot = piece == 0 ? 2 * c0 + 1 : 2 * (c0 + piece);
        pm[k] = p.part_ml[slot * 2 * N + r];
        pl[k] = p.part_ml[(slot * 2 + 1) * N + r];
        const float* o = N == 128 ? p.part_o + slot * N * D + (lane * kPer & ~3) * N + r * 4 + (lane * kPer & 3)
                                  : p.part_o + (slot * N + r) * D + lane * kPer;
        if (D == 128) {
          const float4 x = *reinterpret_cast<const float4*>(o);
          v[k][0] = x.x, v[k][1] = x.y, v[k][kPer - 2] = x.z, v[k][kPer - 1] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(o);
          v[k][0] = x.x, v[k][1] = x.y;
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kStep; ++k) top = fmaxf(top, pm[k]);
      const float old = ex2_approx(m - top);
      m = top;
      sum *= old;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] *= old;
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        if (k0 + k >= pieces) break;
        const float w = ex2_approx(pm[k] - top);
        sum = fmaf(w, pl[k], sum);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, v[k][i], acc[i]);
      }
    }
    if (lane == 0) sm[warp] = m, sl[warp] = sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) so[warp][lane * kPer + i] = acc[i];
    __syncthreads();
    // thread: a channel of one of the block's rows, kRows * D of them over 256 threads
#pragma unroll 1
    for (int x = threadIdx.x; x < kRows * D; x += 256) {
      const int q = x / D, c = x % D, row_r = blockIdx.y * kRows + q;
      float top = sm[q * kW];
#pragma unroll
      for (int k = 1; k < kW; ++k) top = fmaxf(top, sm[q * kW + k]);
      float l = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const float w = ex2_approx(sm[q * kW + k] - top);
        l = fmaf(w, sl[q * kW + k], l);
        y = fmaf(w, so[q * kW + k][c], y);
      }
      if (row_r >= tail[0]) break;
      const int at = tail[3] * N + row_r, t = at / p.group, hq = tail[4] * p.group + at - t * p.group;
      const size_t row = static_cast<size_t>(tail[2] + t) * p.a.Hq + hq;
      static_cast<__nv_bfloat16*>(p.a.out)[row * D + c] = __float2bfloat16(y * (l == 0.f ? 0.f : 1.f / l));
      if (c == 0 && p.a.lse) p.a.lse[row] = l == 0.f ? -INFINITY : (top - kPLog2 + log2f(l)) * kLn2;
    }
  }
  griddep_launch_dependents();
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

// Codes [num_pages * H][page_size][d], one page of one head a box.
bool make_map(CUtensorMap* m, const void* base, const KvCache& c) {
  const EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const cuuint64_t d = c.d, ps = c.page_size;
  cuuint64_t dims[3] = {d, ps, static_cast<cuuint64_t>(c.num_pages) * c.H};
  cuuint64_t strides[2] = {d, d * ps};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(c.d), static_cast<cuuint32_t>(c.page_size), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows a tile: the smallest that holds a KV head's rows of a sequence; 128 is the kernel with the rows on the
// tensor core's rows. 64 sequences, 4 rows a KV head: 174 us with 16, 185 with 32 (d = 64: 146 and 166). 8 sequences
// of up to 16384 tokens: 16 rows 48 and 51 us (d = 64: 46 and 47); 20 and 32 rows 50 and 49 us with 32, 84 and 75 with
// 128 (d = 64: 48 and 46, 76 and 67); 36 and 64 rows 82 and 69 us as one tile of 128, 80 and 68 as two of 32 (d = 64: 74
// and 60, 77 and 63); 16 sequences with 64 query heads a KV head 141 and 136: one tile or two is even there.
int rows_a_tile(const CacheAttnArgs& a) {
  const long long rows = static_cast<long long>(a.Tmax) * (a.Hq / a.cache.H);
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : 128);
}

struct Sizes {
  int N, RT, ctas;
  size_t ml, o, bytes;  // offsets of the partial sums and results
};
Sizes sizes_of(const CacheAttnArgs& a) {
  Sizes s;
  s.N = rows_a_tile(a);
  const long long rows = static_cast<long long>(a.Tmax) * (a.Hq / a.cache.H);
  s.RT = static_cast<int>((rows + s.N - 1) / s.N);
  const long long keys = static_cast<long long>(a.max_pages) * a.cache.page_size;
  const long long units = static_cast<long long>(a.B) * s.RT * a.cache.H * ((keys + 127) / 128);
  s.ctas = static_cast<int>(std::min<long long>(device_sm_count(), units));
  const size_t n = static_cast<size_t>(s.ctas);
  s.ml = (n * 32 + 255) / 256 * 256;
  s.o = s.ml + (n * 2 * 2 * s.N * 4 + 255) / 256 * 256;
  s.bytes = s.o + n * 2 * s.N * a.cache.d * 4;
  return s;
}

template <int D, int N>
cudaError_t launch_t(const CacheAttnArgs& a, const Sizes& z, cudaStream_t st) {
  using C = std::conditional_t<N == 128, Wide<D>, Cfg<D, N == 128 ? 16 : N>>;
  constexpr auto kernel = [] {
    if constexpr (N == 128) return cache_attn_wide_kernel<D>;
    else return cache_attn_kernel<D, N>;
  }();
  Params p;
  if (!make_map(&p.tm_k, a.cache.k, a.cache) || !make_map(&p.tm_v, a.cache.v, a.cache)) return cudaErrorNotSupported;
  p.a = a;
  p.group = a.Hq / a.cache.H;
  p.RT = z.RT;
  p.E = a.B * z.RT;
  p.scale_log2 = a.scale * kLog2e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.tails = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + z.ml);
  p.part_o = reinterpret_cast<float*>(ws + z.o);
  // the shared-memory opt-in is an attribute of the kernel on each device: set once a device
  static std::atomic<unsigned long long> configured[(kMaxDevices + 63) / 64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const bool cacheable = dev >= 0 && dev < kMaxDevices;
  const unsigned long long bit = cacheable ? 1ull << (dev % 64) : 0ull;
  if (!cacheable || !(configured[cacheable ? dev / 64 : 0].load(std::memory_order_acquire) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (cacheable) configured[dev / 64].fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaError_t e = launch_pdl(kernel, dim3(z.ctas), dim3(C::kThreads), C::kSmem, st, p);
  if (e == cudaSuccess && z.ctas > 1)
    e = launch_pdl(cache_attn_join_kernel<D, N>,
                   dim3(z.ctas - 1, (std::min<long long>(N, 1ll * a.Tmax * p.group) + kJoinRows<N> - 1) / kJoinRows<N>),
                   dim3(256), 0, st, p);
  return e;
}

}  // namespace

double cache_attention_units(const CacheAttnArgs& a) {
  const int N = rows_a_tile(a);
  const long long rows = static_cast<long long>(a.Tmax) * (a.Hq / a.cache.H);
  const long long keys = static_cast<long long>(a.max_pages) * a.cache.page_size;
  const long long cost = N == 128 ? kSegCost<128> : kSegCost<16>;
  return static_cast<double>(a.B) * a.cache.H * ((rows + N - 1) / N) * ((keys + 127) / 128 + cost);
}

size_t cache_attention_workspace(const CacheAttnArgs& a) { return sizes_of(a).bytes; }

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st) {
  const Sizes z = sizes_of(a);
  if (a.cache.d == 128)
    return z.N == 16 ? launch_t<128, 16>(a, z, st) : (z.N == 32 ? launch_t<128, 32>(a, z, st) : launch_t<128, 128>(a, z, st));
  return z.N == 16 ? launch_t<64, 16>(a, z, st) : (z.N == 32 ? launch_t<64, 32>(a, z, st) : launch_t<64, 128>(a, z, st));
}

cudaError_t read_cache_attn_error(cudaStream_t st, int clear, int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_cache_attn_error, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e != cudaSuccess) return e;
  if ((e = cudaStreamSynchronize(st)) != cudaSuccess) return e;
  if (clear && v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_cache_attn_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (code) *code = v;
  return e;
}

}  // namespace fpattn
