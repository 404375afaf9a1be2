// Shared pieces of the 8-bit paged cache's kernels (append, attention).
//
// A page holds `page` tokens of every head as e4m3 values, [H][page][d], and
// one fp32 scale per head for its keys and one for its values; a stored value
// x stands for x * scale.  Scales are powers of two: e4m3 is a floating-point
// format, so a power of two loses nothing against an exact one but the last
// fraction of a binade of range, dividing by it is exact, and its logarithm
// is an integer that folds into the softmax exponent.
#pragma once

#include "common.cuh"

namespace pp {

// Exponents a scale may have.  The attention kernels carry a page's value
// scale inside the exponent (2^(s + log2 scale - M)), so two pages' scales
// must not differ by more than a softmax term's fp32 range allows: 80 of the
// 126 binades below 1, which leaves probabilities down to 2^-46.
constexpr int kScaleMinExp = -40, kScaleMaxExp = 40;

// Smallest power of two 2^e with amax <= 448 * 2^e, e clamped; 448 =
// 1.75 * 2^8 is e4m3's largest value.  amax finite, >= 0.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = e < kScaleMinExp ? kScaleMinExp : e > kScaleMaxExp ? kScaleMaxExp : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two floats -> two e4m3 bytes (a in the low byte), round to nearest even,
// out of range saturates to +-448, NaN stays NaN (0x7f).
__device__ __forceinline__ uint32_t f2_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two e4m3 bytes (the low 16 bits of w) -> f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_h2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t w) {
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f2_to_h2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// Table entry -> page, or -1 when the entry names none.
__device__ __forceinline__ int page_of(int32_t entry, int n_pages) {
  return (uint32_t)entry < (uint32_t)n_pages ? entry : -1;
}

// The document pass's split plan gives every unit this many steps ahead of its
// tiles: what a run costs beside them (queries in, partial result out: about
// 14000 cycles, a tile 3450), so that a CTA whose range meets a unit's border
// gets fewer tiles.  They hold no tile: the unit's first chunk is that of the
// CTA of step kKv8Lead.
constexpr int kKv8Lead = 4;

// A run of tiles of one unit, (key head, row group), in a CTA of the document pass.
// Steps are counted in 32 bits (the host keeps W, and C times a remainder by C, below
// 2^31), and only a CTA's first run divides: 64-bit divisions at every role's start
// took 3600 cycles.
struct Seg8 {
  int u, h, gi, j0, n;
  bool two;     // two M tiles; else one, its tiles dealt out to the streams
};
struct Runs8 {
  int t, t_end, u, h, gi;
};
__host__ __device__ __forceinline__ Runs8 first_run8(const SplitPlan& p, int cta) {
  Runs8 r;
  const int q = (int)p.W / p.C, m = (int)p.W - q * p.C;   // floor(cta W / C)
  r.t = cta * q + cta * m / p.C;
  r.t_end = (cta + 1) * q + (cta + 1) * m / p.C;
  r.u = r.t / p.T;
  r.h = r.u / p.G;
  r.gi = r.u - r.h * p.G;
  return r;
}
// rows: (query row, query head) pairs of a key head.
__host__ __device__ __forceinline__ bool next_seg8(const SplitPlan& p, int rows, Runs8& r,
                                                   Seg8& s) {
  while (r.t < r.t_end) {
    s.u = r.u;
    s.h = r.h;
    s.gi = r.gi;
    s.two = rows - s.gi * kGroupRows > 128;
    const int v = r.t - r.u * p.T;              // step of the unit
    const int n = p.T - v < r.t_end - r.t ? p.T - v : r.t_end - r.t;
    r.t += n;
    if (v + n == p.T) {
      ++r.u;
      if (++r.gi == p.G) {
        r.gi = 0;
        ++r.h;
      }
    }
    s.j0 = v > kKv8Lead ? v - kKv8Lead : 0;
    s.n = v + n - kKv8Lead - s.j0;
    if (s.n > 0) return true;
  }
  return false;
}
// The first tile of stream st (0, 1) in a run, and whether it has one: a run of one
// tile of one M tile leaves stream 1 without.  Such a stream takes no part in the
// run's barriers: nothing would hold its warps back before their next run's arrival,
// and a barrier two phases on looks to its waiter like one that has not moved.
__host__ __device__ __forceinline__ int first_tile8(const Seg8& s, int st) {
  return s.two ? 0 : st;
}
__host__ __device__ __forceinline__ bool has_tile8(const Seg8& s, int st) {
  return first_tile8(s, st) < s.n;
}

// How the segment pass groups (query row, query head) pairs that share a key head
// into a warp's item.  A decode step's rows belong to different streams, an item
// each; question rows share their segment, so 16 pairs go together, unless that
// makes fewer items than the GPU holds warps at a time: then 8 do, which a warp
// finishes sooner (64 questions of 32 rows, 8 heads: 53 us by 16, 36 by 8; 64 of
// 30, 32 heads, 8000 keys: 289 and 318).
struct Kv8Items {
  int most, hg, gt, rt;   // pairs at most, heads, items per key head's group, rows
  int64_t items;
};
constexpr int kFewItems = 12 * 148;
inline Kv8Items kv8_items(int rows, int g, int H, bool one_row_per_stream) {
  Kv8Items x;
  for (x.most = one_row_per_stream && g <= 8 ? 8 : 16;; x.most = 8) {
    x.hg = g < x.most ? g : x.most;
    x.gt = (g + x.hg - 1) / x.hg;
    x.rt = one_row_per_stream ? 1 : x.most / x.hg;
    x.items = (int64_t)((rows + x.rt - 1) / x.rt) * H * x.gt;
    if (x.most == 8 || x.items >= kFewItems) return x;
  }
}

}  // namespace pp
