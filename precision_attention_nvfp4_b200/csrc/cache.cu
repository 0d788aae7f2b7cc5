// Rotary positions and the FP8 KV cache: rotate, quantise on the way in, read
// back. All three are streams of bf16 rows and bound by memory; a thread
// keeps two 16-byte chunks of a row, chosen so that both channels of every
// rotated pair are its own and that a load covers neighbouring chunks.
//
// Rows are d channels, d / 16 threads a row. With the half layout thread j of
// a row takes chunks j and j + dim / 16 (channel i and its partner i + dim / 2),
// those past them two chunks of the part that is not rotated; with the
// interleaved one chunks j and j + d / 16, whose pairs lie within a chunk. A
// group of d / 16 threads stays with one token and walks over its heads, so sine
// and cosine are worked out once a token and group and used for every head;
// the loads of kBatch rows are issued before any of them is worked on.
//
// Angles: the table holds the turns a position as 64-bit fractions, so
// position * turns in wrapping integer arithmetic is the angle modulo a turn
// (to 2^-63 |position| turns), where fp32 angles lose 2^-24 |angle|. The
// top 32 bits are split into a quadrant and a remainder within an eighth of a
// turn, whose sine and cosine are Taylor sums (truncated below 3e-8).
#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>

#include "serve_internal.h"
#include "sm100.cuh"

namespace fpattn {

namespace {

constexpr int kCacheThreads = 128;
constexpr int kMinExp = -63;
// Rows a thread has in flight: the prefill write takes 76.4 us with 4, 85.9 with 2, 76.8 with 8; the rotary gradient 26.1,
// 29.3 and 26.1.
constexpr int kBatch = 4;


__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}
__device__ __forceinline__ void unpack(const uint4& v, float* f) {
  f[0] = lo_bf16(v.x); f[1] = hi_bf16(v.x);
  f[2] = lo_bf16(v.y); f[3] = hi_bf16(v.y);
  f[4] = lo_bf16(v.z); f[5] = hi_bf16(v.z);
  f[6] = lo_bf16(v.w); f[7] = hi_bf16(v.w);
}
__device__ __forceinline__ uint4 pack(const float* f) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Sine and cosine, times m, of position * turns.
__device__ __forceinline__ void sincos_turns(unsigned long long pos, unsigned long long turns, float m, float& s,
                                             float& c) {
  const uint32_t x = static_cast<uint32_t>((pos * turns) >> 32);
  const uint32_t quad = (x + 0x20000000u) >> 30;
  const int r = static_cast<int>(x - (quad << 30));              // [-2^29, 2^29): an eighth of a turn either way
  const float t = static_cast<float>(r) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float t2 = t * t;
  float sn = fmaf(t2, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(sn, t2, 8.3333333e-3f);
  sn = fmaf(sn, t2, -1.6666667e-1f);
  sn = fmaf(sn * t2, t, t);
  float cs = fmaf(t2, 2.4801587e-5f, -1.3888889e-3f);
  cs = fmaf(cs, t2, 4.1666667e-2f);
  cs = fmaf(cs, t2, -0.5f);
  cs = fmaf(cs, t2, 1.0f);
  const float a = (quad & 1u) ? cs : sn, b = (quad & 1u) ? sn : cs;
  s = m * ((quad & 2u) ? -a : a);
  c = m * (((quad + 1u) & 2u) ? -b : b);
}

// The same in 64 bits. Taylor sums to t^13 and t^12, truncated below 4e-13.
__device__ __forceinline__ void sincos_turns(unsigned long long pos, unsigned long long turns, float m, double& s,
                                             double& c) {
  const unsigned long long x = pos * turns;
  const uint32_t quad = static_cast<uint32_t>((x + 0x2000000000000000ull) >> 62);
  const double t = static_cast<double>(static_cast<long long>(x - (static_cast<unsigned long long>(quad) << 62))) *
                   3.4061215800865545e-19;  // 2 pi / 2^64
  const double t2 = t * t;
  double sn = fma(t2, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  sn = fma(sn, t2, 1.0 / 362880.0);
  sn = fma(sn, t2, -1.0 / 5040.0);
  sn = fma(sn, t2, 1.0 / 120.0);
  sn = fma(sn, t2, -1.0 / 6.0);
  sn = fma(sn * t2, t, t);
  double cs = fma(t2, 1.0 / 479001600.0, -1.0 / 3628800.0);
  cs = fma(cs, t2, 1.0 / 40320.0);
  cs = fma(cs, t2, -1.0 / 720.0);
  cs = fma(cs, t2, 1.0 / 24.0);
  cs = fma(cs, t2, -0.5);
  cs = fma(cs, t2, 1.0);
  const double a = (quad & 1u) ? cs : sn, b = (quad & 1u) ? sn : cs;
  s = m * ((quad & 2u) ? -a : a);
  c = m * (((quad + 1u) & 2u) ? -b : b);
}

// Read or written once: kept out of the way of what others keep in cache.
__device__ __forceinline__ uint4 load_row(const uint4* p) { return __ldcs(p); }
__device__ __forceinline__ void store_row(uint4* p, const uint4& v) { __stcs(p, v); }

// The two 16-byte chunks of a row that thread j keeps, and whether they rotate.
struct Place {
  int a, b;
  bool ta, tb;
};
template <int D>
__device__ __forceinline__ Place place_of(int j, int dim, int interleaved) {
  constexpr int kLanes = D / 16;
  if (interleaved) return {j, j + kLanes, j < (dim >> 3), j + kLanes < (dim >> 3)};
  const int turning = dim >> 4;
  if (j < turning) return {j, j + turning, true, true};
  const int first = 2 * turning + (j - turning);
  return {first, first + kLanes - turning, false, false};
}

// Sine and cosine of the eight pairs of thread j at a position; identity where a chunk does not rotate.
__device__ __forceinline__ void pair_angles(const RotaryTable& tab, const Place& pl, int j, long long position, float (&sn)[8],
                                            float (&cs)[8]) {
  const unsigned long long pos = static_cast<unsigned long long>(position);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sn[i] = 0.f;
    cs[i] = 1.f;
    if (i < 4 ? pl.ta : pl.tb) {
      const int pair = tab.interleaved ? 4 * (i < 4 ? pl.a : pl.b) + (i & 3) : 8 * j + i;
      sincos_turns(pos, tab.turns[pair], tab.magnitude, sn[i], cs[i]);
    }
  }
}

// f[0..8) and f[8..16) are the chunks a and b. Pairs: half layout (f[i],
// f[8 + i]), interleaved (f[2 i], f[2 i + 1]).
__device__ __forceinline__ void turn_row(float (&f)[16], const float (&sn)[8], const float (&cs)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = f[2 * i], y = f[2 * i + 1];
      f[2 * i] = fmaf(x, cs[i], -(y * sn[i]));
      f[2 * i + 1] = fmaf(x, sn[i], y * cs[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = f[i], y = f[8 + i];
      f[i] = fmaf(x, cs[i], -(y * sn[i]));
      f[8 + i] = fmaf(x, sn[i], y * cs[i]);
    }
  }
}

// Rounded to the odd neighbour where it is not exact: a later rounding to fewer bits gives what it would have given.
__device__ __forceinline__ float to_odd(double x) {
  const float f = __double2float_rz(x);
  return static_cast<double>(f) == x || !(fabsf(f) < INFINITY) ? f : __uint_as_float(__float_as_uint(f) | 1u);
}
// A rotated pair in 64 bits.
__device__ __noinline__ float2 turned_pair(float x, float y, long long pos, unsigned long long turns, float m) {
  double s, c;
  sincos_turns(static_cast<unsigned long long>(pos), turns, m, s, c);
  const double a = x, b = y;
  return make_float2(to_odd(fma(a, c, -(b * s))), to_odd(fma(a, s, b * c)));
}

// Largest |f| of the row whose D / 16 threads call together, as an integer: its order is that of the floats, and a NaN is
// above infinity.
template <int kLanes>
__device__ __forceinline__ uint32_t row_amax(const float (&f)[16]) {
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}
// The smallest e >= kMinExp with A <= 448 * 2^e = 1.75 * 2^(e + 8): a mantissa above .75 carries into the exponent.
__device__ __forceinline__ int row_exp(uint32_t a) { return max(kMinExp, static_cast<int>((a + 0x1FFFFFu) >> 23) - 135); }
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return static_cast<uint32_t>(cvt_e4m3x2(a, b)) | static_cast<uint32_t>(cvt_e4m3x2(c, d)) << 16;
}

struct RotaryParams {
  const uint4* x;
  uint4* out;
  long long xb, xt, xh, ob, ot, oh;  // strides in 16-byte chunks
  int T, H, heads;                   // heads: of a token, per group of threads
  long long tokens;                  // B * T
  const long long* positions;
  int per_b;
  int transpose;
  RotaryTable tab;
};

// A group of D / 16 threads takes one token and p.heads of its heads.
// Bound by memory: 4 bytes a channel; 4 x 4096 tokens of 32 heads, d = 128: 43 us,
// 6.3 TB/s; the transpose of 32 of 64 channels, 15003 tokens of 40 heads: 27.6 us, 5.6 TB/s
// (26.2 us in a replayed graph).
template <int D>
__global__ void __launch_bounds__(kCacheThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kLanes = D / 16;
  griddep_wait();
  const long long tok = static_cast<long long>(blockIdx.x) * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
  if (tok < p.tokens) {
    const int j = threadIdx.x % kLanes;
    const Place pl = place_of<D>(j, p.tab.dim, p.tab.interleaved);
    const int b = static_cast<int>(tok / p.T), t = static_cast<int>(tok - static_cast<long long>(b) * p.T);
    const int h0 = blockIdx.y * p.heads, h1 = min(p.H, h0 + p.heads);
    const uint4* x = p.x + b * p.xb + t * p.xt;
    uint4* o = p.out + b * p.ob + t * p.ot;
    float sn[8], cs[8];
    const long long pos = p.positions[p.per_b ? tok : t];
    for (int h = h0; h < h1; h += kBatch) {
      uint4 va[kBatch], vb[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (h + k >= h1) break;
        va[k] = load_row(x + (h + k) * p.xh + pl.a);
        vb[k] = load_row(x + (h + k) * p.xh + pl.b);
      }
      if (h == h0 && (pl.ta || pl.tb)) {  // behind the first loads
        pair_angles(p.tab, pl, j, pos, sn, cs);
        if (p.transpose) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (h + k >= h1) break;
        if (pl.ta || pl.tb) {
          float f[16];
          unpack(va[k], f);
          unpack(vb[k], f + 8);
          turn_row(f, sn, cs, p.tab.interleaved);
          va[k] = pack(f);
          vb[k] = pl.tb ? pack(f + 8) : vb[k];
        }
        store_row(o + (h + k) * p.oh + pl.a, va[k]);
        store_row(o + (h + k) * p.oh + pl.b, vb[k]);
      }
    }
  }
  griddep_launch_dependents();
}

struct WriteParams {
  const uint4 *k, *v, *q;
  uint4* q_out;
  long long kt, kh, vt, vh, qt, qh, ot, oh;  // strides in 16-byte chunks
  int T, H, Hq, rows, per;                   // rows of a token: 2 H + Hq; per: of them, per group of threads
  const long long* slots;
  const long long* positions;
  RotaryTable tab;
  KvCache cache;
  int* nonfinite;
};

enum : int { kPlain, kHalf, kInterleaved };  // is K rotated, and how

// Row r of a token: K head r, V head r - H, Q head r - 2 H.
// Bound by memory: 3 bytes a channel of K and V, 4 of Q; 15361 tokens of 8 KV and
// 32 query heads, d = 128: 77 us, 4.5 TB/s; 68 without the second look at K's
// values beside a rounding boundary, 93 with all of K's in 64 bits. Without
// rotation (K and V alone) 22.7 us, 4.1 TB/s. The layout is a parameter of the
// kernel: one kernel for all took 93 and 33 us (142 registers, 3 blocks an SM).
template <int D, int kLayout>
__global__ void __launch_bounds__(kCacheThreads, 4) cache_write_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kLanes = D / 16;
  constexpr bool inter = kLayout == kInterleaved;
  griddep_wait();
  const int tok = blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
  // every thread stays for the shuffles below; a token past the end is read as the last one and written nowhere
  const bool live = tok < p.T;
  const long long t = live ? tok : p.T - 1;
  const int j = threadIdx.x % kLanes;
  const Place pl = place_of<D>(j, p.tab.dim, inter);
  const bool turn = kLayout != kPlain && (pl.ta || pl.tb);
  const long long pos = kLayout != kPlain ? p.positions[t] : 0;
  const long long slot = p.slots[t];
  const int page_log = 31 - __clz(p.cache.page_size);
  const long long page = slot >> page_log;
  const int off = static_cast<int>(slot) & (p.cache.page_size - 1);
  const bool store = live && slot >= 0 && page < p.cache.num_pages;
  const int r0 = blockIdx.y * p.per, r1 = min(p.rows, r0 + p.per);
  float sn[8], cs[8];
  for (int r = r0; r < r1; r += kBatch) {
    uint4 va[kBatch], vb[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r + k >= r1) break;
      const int h = r + k;
      const uint4* src = h >= 2 * p.H ? p.q + t * p.qt + (h - 2 * p.H) * p.qh
                                      : (h >= p.H ? p.v + t * p.vt + (h - p.H) * p.vh : p.k + t * p.kt + h * p.kh);
      va[k] = load_row(src + pl.a);
      vb[k] = load_row(src + pl.b);
    }
    // behind the first loads; a group of V rows alone needs none
    if (r == r0 && turn && (r0 < p.H || r1 > 2 * p.H)) pair_angles(p.tab, pl, j, pos, sn, cs);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r + k >= r1) break;
      const bool is_q = r + k >= 2 * p.H, is_v = !is_q && r + k >= p.H;
      const int h = is_q ? r + k - 2 * p.H : (is_v ? r + k - p.H : r + k);
      float f[16];
      unpack(va[k], f);
      unpack(vb[k], f + 8);
      if (turn && !is_v) turn_row(f, sn, cs, inter);
      if (is_q) {
        if (live) {
          uint4* o = p.q_out + t * p.ot + h * p.oh;
          o[pl.a] = pack(f);
          o[pl.b] = pl.tb ? pack(f + 8) : vb[k];
        }
        continue;
      }
      uint32_t a = row_amax<kLanes>(f);
      int e = row_exp(a);
      float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e <= 120
      uint32_t w[4];
      if (kLayout != kPlain && !is_v) {  // (the same for the whole warp, as the votes below need)
        // fp32 angles and products leave a pair off by less than 2^-21 (|x| + |y|) m, at most 2^-20 of its larger result.
        // Pairs of which that decides a code (one element in 10000) are rotated again in 64 bits, and so is every pair
        // of a row of whose exponent it decides (8 rows in a million).
        const bool edge = a > 17u && row_exp(a - 17u) != row_exp(a + 17u);
        const float off = up * 9.6e-7f;  // 2^-20, and a little for the rounding of what it is added to
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          d[i] = (i < 4 ? pl.ta : pl.tb)
                     ? off * fmaxf(fabsf(inter ? f[2 * i] : f[i]), fabsf(inter ? f[2 * i + 1] : f[8 + i]))
                     : 0.f;
        uint32_t differ[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d0 = d[inter ? 2 * i : (4 * i) & 7], d1 = d[inter ? 2 * i : (4 * i + 1) & 7];
          const float d2 = d[inter ? 2 * i + 1 : (4 * i + 2) & 7], d3 = d[inter ? 2 * i + 1 : (4 * i + 3) & 7];
          const float* g = f + 4 * i;
          w[i] = codes4(fmaf(g[0], up, d0), fmaf(g[1], up, d1), fmaf(g[2], up, d2), fmaf(g[3], up, d3));
          differ[i] = w[i] ^ codes4(fmaf(g[0], up, -d0), fmaf(g[1], up, -d1), fmaf(g[2], up, -d2), fmaf(g[3], up, -d3));
        }
        if ((differ[0] | differ[1] | differ[2] | differ[3] | (edge ? 1u : 0u)) && a < 0x7F800000u) {
          float x[16];
          unpack(va[k], x);
          unpack(vb[k], x + 8);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t here = inter ? differ[i >> 1] >> (16 * (i & 1)) & 0xFFFFu
                                        : (differ[i >> 2] | differ[2 + (i >> 2)]) >> (8 * (i & 3)) & 0xFFu;
            if ((here || edge) && (i < 4 ? pl.ta : pl.tb)) {
              const int pair = inter ? 4 * (i < 4 ? pl.a : pl.b) + (i & 3) : 8 * j + i;
              const float2 y = turned_pair(inter ? x[2 * i] : x[i], inter ? x[2 * i + 1] : x[8 + i], pos, p.tab.turns[pair],
                                           p.tab.magnitude);
              if (inter) f[2 * i] = y.x, f[2 * i + 1] = y.y;
              else f[i] = y.x, f[8 + i] = y.y;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = codes4(f[4 * i] * up, f[4 * i + 1] * up, f[4 * i + 2] * up, f[4 * i + 3] * up);
        }
        if (__any_sync(0xffffffffu, edge)) {
          a = row_amax<kLanes>(f);
          if (edge) {
            e = row_exp(a);
            up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = codes4(f[4 * i] * up, f[4 * i + 1] * up, f[4 * i + 2] * up, f[4 * i + 3] * up);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = codes4(f[4 * i] * up, f[4 * i + 1] * up, f[4 * i + 2] * up, f[4 * i + 3] * up);
      }
      const bool bad = a >= 0x7F800000u;
      if (bad) w[0] = w[1] = w[2] = w[3] = 0u;
      if (store) {
        const long long row = page * p.H + h;
        uint8_t* codes = (is_v ? p.cache.v : p.cache.k) + ((row << page_log) + off) * D;
        *reinterpret_cast<uint2*>(codes + 8 * pl.a) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(codes + 8 * pl.b) = make_uint2(w[2], w[3]);
        if (j == 0) {
          p.cache.exps[((2 * row + (is_v ? 1 : 0)) << page_log) + off] = bad ? 255 : static_cast<uint8_t>(e + 127);
          if (bad && p.nonfinite) atomicExch(p.nonfinite, 1);
        }
      }
    }
  }
  griddep_launch_dependents();
}

// 67.4 us in a replayed graph against 68.9 with four (prefix of 65536 tokens, 8 heads, d = 128).
constexpr int kReadBatch = 8;

struct ReadParams {
  uint4 *k, *v;
  long long kt, kh, vt, vh;
  int T, H, per;
  const long long* slots;
  KvCache cache;
};

// Two E4M3 codes times 2^e as packed bf16. A code has 4 bits, so the product
// is exact unless it passes bf16's range; kept at its largest there.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t two, float scale) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two)));
  const __half2 h = *reinterpret_cast<__half2*>(&h2);
  const float2 f = __half22float2(h);
  constexpr float kMax = 3.3895313892515355e38f;
  const float x = f.x * scale, y = f.y * scale;
  // a NaN scale has to stay: fminf and fmaxf would drop it
  return pack_bf16(fabsf(x) > kMax ? copysignf(kMax, x) : x, fabsf(y) > kMax ? copysignf(kMax, y) : y);
}

// Thread j of a row takes codes 16 j .. 16 j + 15.
// Bound by memory: 3 bytes a channel; 65536 tokens of 8 heads, d = 128: 71.5 us, 5.6 TB/s
// (67.4 us, 6.0 TB/s, in a replayed graph).
template <int D>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kLanes = D / 16;
  griddep_wait();
  const int tok = blockIdx.x * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
  if (tok < p.T) {
    const int j = threadIdx.x % kLanes;
    const long long t = tok;
    const long long slot = p.slots[t];
    const int page_log = 31 - __clz(p.cache.page_size);
    const long long page = slot >> page_log;
    const int off = static_cast<int>(slot) & (p.cache.page_size - 1);
    const bool there = slot >= 0 && page < p.cache.num_pages;
    const int r0 = blockIdx.y * p.per, r1 = min(2 * p.H, r0 + p.per);
    for (int r = r0; r < r1; r += kReadBatch) {
      uint4 c[kReadBatch];
      uint32_t e[kReadBatch];
#pragma unroll
      for (int k = 0; k < kReadBatch; ++k) {
        c[k] = make_uint4(0u, 0u, 0u, 0u);
        e[k] = 127u;
        if (r + k < r1 && there) {
          const bool is_v = r + k >= p.H;
          const long long row = page * p.H + (is_v ? r + k - p.H : r + k);
          c[k] = load_row(reinterpret_cast<const uint4*>((is_v ? p.cache.v : p.cache.k) + ((row << page_log) + off) * D + 16 * j));
          e[k] = p.cache.exps[((2 * row + (is_v ? 1 : 0)) << page_log) + off];
        }
      }
#pragma unroll
      for (int k = 0; k < kReadBatch; ++k) {
        if (r + k >= r1) break;
        const bool is_v = r + k >= p.H;
        const int h = is_v ? r + k - p.H : r + k;
        // byte 255 stands for NaN; 2^-127 (byte 0, which this library does not write) is subnormal
        const float scale = e[k] == 255u ? __uint_as_float(0x7FC00000u)
                                         : (e[k] == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e[k] << 23));
        const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] = codes_to_bf16(w[i] & 0xFFFFu, scale);
          o[2 * i + 1] = codes_to_bf16(w[i] >> 16, scale);
        }
        uint4* dst = is_v ? p.v + t * p.vt + h * p.vh : p.k + t * p.kt + h * p.kh;
        store_row(dst + 2 * j, make_uint4(o[0], o[1], o[2], o[3]));
        store_row(dst + 2 * j + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
  griddep_launch_dependents();
}

// Rows of a token that a group of threads takes: kRowsMost of them once there
// are tokens enough (one set of angles serves them, and the last wave of short
// blocks is a small part), fewer when there are not, so that the card is filled.
// With 2, 4, 8, 16 and 32 at most the prefill write takes 107, 82, 76, 77 and 77 us, the
// read of a prefix 106, 82, 67, 70 and 70. Threads to fill the card with, 148 times 512,
// 1024, 2048 and 4096: the same for many tokens, a write of 1000 tokens 8.2, 7.7, 8.6
// and 12.4 us, 15361 tokens of d = 64 40.0, 40.0, 40.3 and 46.6.
constexpr int kRowsMost = 8;
int rows_per_group(long long tokens, int lanes, int rows) {
  const long long want = 148ll * 2048;  // threads
  const long long groups = (want + tokens * lanes - 1) / (tokens * lanes);
  const long long per = (rows + groups - 1) / groups;
  return static_cast<int>(per < kRowsMost ? per : kRowsMost);
}

}  // namespace

cudaError_t launch_rotary(const Rows& x, const RotaryTable& tab, const long long* positions, bool per_b,
                          bool transpose, const Rows& out, cudaStream_t st) {
  RotaryParams p;
  p.x = static_cast<const uint4*>(x.data);
  p.out = static_cast<uint4*>(out.data);
  p.xb = x.sb / 8, p.xt = x.st / 8, p.xh = x.sh / 8;
  p.ob = out.sb / 8, p.ot = out.st / 8, p.oh = out.sh / 8;
  p.T = x.T;
  p.H = x.H;
  p.tokens = static_cast<long long>(x.B) * x.T;
  p.positions = positions;
  p.per_b = per_b;
  p.transpose = transpose;
  p.tab = tab;
  const int lanes = x.d / 16, groups = kCacheThreads / lanes;
  p.heads = rows_per_group(p.tokens, lanes, x.H);
  const dim3 grid(static_cast<unsigned>((p.tokens + groups - 1) / groups), (x.H + p.heads - 1) / p.heads);
  return launch_pdl(x.d == 128 ? rotary_kernel<128> : rotary_kernel<64>, grid, dim3(kCacheThreads), 0, st, p);
}

cudaError_t launch_cache_write(const KvCache& c, const Rows& k, const Rows& v, const long long* slots,
                               const RotaryTable& tab, const long long* positions, const Rows* q, const Rows* q_out,
                               int* nonfinite, cudaStream_t st) {
  WriteParams p{};
  p.k = static_cast<const uint4*>(k.data);
  p.v = static_cast<const uint4*>(v.data);
  p.kt = k.st / 8, p.kh = k.sh / 8, p.vt = v.st / 8, p.vh = v.sh / 8;
  p.T = k.T;
  p.H = k.H;
  if (q) {
    p.q = static_cast<const uint4*>(q->data);
    p.q_out = static_cast<uint4*>(q_out->data);
    p.qt = q->st / 8, p.qh = q->sh / 8, p.ot = q_out->st / 8, p.oh = q_out->sh / 8;
    p.Hq = q->H;
  }
  p.rows = 2 * p.H + p.Hq;
  p.slots = slots;
  p.positions = positions;
  p.tab = tab;
  p.cache = c;
  p.nonfinite = nonfinite;
  const int lanes = c.d / 16, groups = kCacheThreads / lanes;
  p.per = rows_per_group(p.T, lanes, p.rows);
  const dim3 grid((p.T + groups - 1) / groups, (p.rows + p.per - 1) / p.per);
  auto pick = [&](auto plain, auto half, auto interleaved) {
    return tab.dim == 0 ? plain : (tab.interleaved ? interleaved : half);
  };
  auto kernel = c.d == 128 ? pick(cache_write_kernel<128, kPlain>, cache_write_kernel<128, kHalf>,
                                  cache_write_kernel<128, kInterleaved>)
                           : pick(cache_write_kernel<64, kPlain>, cache_write_kernel<64, kHalf>,
                                  cache_write_kernel<64, kInterleaved>);
  return launch_pdl(kernel, grid, dim3(kCacheThreads), 0, st, p);
}

cudaError_t launch_cache_read(const KvCache& c, const long long* slots, const Rows& k, const Rows& v,
                              cudaStream_t st) {
  ReadParams p{};
  p.k = static_cast<uint4*>(k.data);
  p.v = static_cast<uint4*>(v.data);
  p.kt = k.st / 8, p.kh = k.sh / 8, p.vt = v.st / 8, p.vh = v.sh / 8;
  p.T = k.T;
  p.H = k.H;
  p.slots = slots;
  p.cache = c;
  const int lanes = c.d / 16, groups = kCacheThreads / lanes;
  p.per = rows_per_group(p.T, lanes, 2 * p.H);
  const dim3 grid((p.T + groups - 1) / groups, (2 * p.H + p.per - 1) / p.per);
  return launch_pdl(c.d == 128 ? cache_read_kernel<128> : cache_read_kernel<64>, grid, dim3(kCacheThreads), 0, st, p);
}

}  // namespace fpattn
