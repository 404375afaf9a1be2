// Append to the 8-bit paged cache: rotate keys (and queries) by position,
// quantise keys and values to e4m3, one launch.
//
// Row i of stream s at position p goes to slot p (document, s = 0) or
// p - pos0 (answer stream) of that stream's pages, so the call reads no
// lengths and a repeated call writes the same bytes.  Per (page, head):
//     A = max |x| over the call's rows in the page, need = 2^ceil(log2(A/448))
//     scale = need                when the rows begin at the page's slot 0
//           = max(old, need)      otherwise; the slots before the first row
//                                 are rounded again when the scale grew
//     stored = rn_e4m3(x / scale)
// The rows of one page must be quantised together, so the call's rows of a
// stream stand next to each other at consecutive positions (a question's or a
// document's rows do): the rows of a page are then a run, its first row -- the
// leader -- is found from its neighbour alone, and the leader's warps own the
// page's heads without any ordering between CTAs.  A row that breaks the run is a
// leader too; its scan of the earlier stream ids finds it out, and it is dropped
// with the rest of its page.
//
// Bound: HBM (bf16 in, e4m3 out); a decode step's few kilobytes a row are
// latency.
#include <atomic>

#include "kv8.cuh"
#include "internal.h"
#include "warp_mma.cuh"

namespace pp {
namespace {

struct AppendParams {
  pp_kv8_layer L;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_ld, v_ld, q_ld, qo_ld;   // elements between rows
  int Hq, n;
  const int16_t* sid;
  const int32_t* pos;
  const float* cos_sin;              // [max_pos][rot]: rot/2 cosines, rot/2 sines
  int rot, interleaved, max_pos;     // rot 0: no rotation
  int win;                           // rows whose leaders one CTA looks after, at most 32
  int ys;                            // CTAs along y for keys and values; the rest turn queries
};

// A lane's eight dims of a row, as two groups of four: dims that turn together
// are a lane's own (j and j + rot/2, or neighbours when interleaved), so no
// value crosses lanes and a lane needs four angles.
struct LaneDims {
  int a, b;        // first dims of the groups
  bool turns;
};
template <bool INTER>
__device__ __forceinline__ LaneDims lane_dims(const AppendParams& p, int u) {
  const int hr = p.rot >> 3;              // lanes whose dims turn
  const bool split = u < hr && !INTER;
  return {split ? u * 4 : u * 8, split ? (u + hr) * 4 : u * 8 + 4, u < hr};
}

// Two groups of four bf16 -> floats.
__device__ __forceinline__ void unpack8(uint2 a, uint2 b, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 f = bf2_to_f2(w[c]);
    x[2 * c] = f.x;
    x[2 * c + 1] = f.y;
  }
}

// Turn the lane's dims by the angles' cosines and sines; INTER: neighbours turn together (known
// when compiled: selecting at run time doubled the rotation's instructions).  Every product and difference is
// rounded by itself (no fused multiply-add), the result a plain fp32 evaluation
// of a cos - b sin gives, so which e4m3 value a rotated key rounds to does not
// depend on the compiler's contraction.
template <bool INTER>
__device__ __forceinline__ void turn8(const float4 c4, const float4 s4, float (&x)[8]) {
  const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
  float y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float a = INTER ? x[2 * e] : x[e], b = INTER ? x[2 * e + 1] : x[4 + e];
    y[e] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
    y[4 + e] = __fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e]));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = INTER ? y[(e & 1) * 4 + (e >> 1)] : y[e];
    x[4 + e] = INTER ? y[(e & 1) * 4 + 2 + (e >> 1)] : y[4 + e];
  }
}

// The same by position pos, from the table.
template <bool INTER>
__device__ __forceinline__ void turn8_at(const AppendParams& p, int pos, int u, float (&x)[8]) {
  const float* t = p.cos_sin + (int64_t)pos * p.rot + u * 4;
  turn8<INTER>(__ldg(reinterpret_cast<const float4*>(t)),
               __ldg(reinterpret_cast<const float4*>(t + (p.rot >> 1))), x);
}

// Largest finite magnitude of 8 values, joined to a; any non-finite: bad.
__device__ __forceinline__ void amax8(const float (&x)[8], float& a, bool& bad) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = fabsf(x[e]);
    const bool fin = y < INFINITY;
    a = fmaxf(a, fin ? y : 0.f);
    bad |= !fin;
  }
}

// 4 values over a power-of-two scale -> 4 e4m3 bytes.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float inv) {
  return f2_to_e4m3x2(a * inv, b * inv) | (f2_to_e4m3x2(c * inv, d * inv) << 16);
}

// The slots [0, n) of one head's page (n * d bytes), rounded again after its
// scale grew: x -> rn_e4m3(x * ratio), ratio = old / new < 1; thread t of nt.
template <int D>
__device__ __forceinline__ void requant(uint8_t* base, int n, float ratio, int t, int nt) {
  for (int c = t; c < n * (D / 16); c += nt) {
    uint4* at = reinterpret_cast<uint4*>(base) + c;
    const uint4 w = *at;
    uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 lo = h2_to_f2(e4m3x2_to_h2(a[i])), hi = h2_to_f2(e4m3x2_hi_to_h2(a[i]));
      a[i] = f2_to_e4m3x2(lo.x * ratio, lo.y * ratio) |
             (f2_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
    }
    *at = make_uint4(a[0], a[1], a[2], a[3]);
  }
}

// A lane's 8 dims of a row's key and value to the row at k_row, v_row.  All lanes
// call it.
template <int D>
__device__ __forceinline__ void put8(uint8_t* k_row, uint8_t* v_row, const LaneDims& ld, int u,
                                     bool on, const float (&kx)[8], float (&vx)[8], float ki,
                                     float vi, bool bad, int lane) {
  constexpr int U = D / 8;
  uint32_t nan_lanes = 0;
  if (bad) {
    // A NaN among a row's values is kept by its key: value 0, first key element
    // NaN.  Queries that see the row come out NaN either way, and queries that
    // do not see it are not touched by 0 * NaN.
    bool vn = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool n = vx[e] != vx[e];
      vn |= n;
      vx[e] = n ? 0.f : vx[e];
    }
    nan_lanes = __ballot_sync(0xffffffffu, vn);
  }
  uint32_t k0 = quant4(kx[0], kx[1], kx[2], kx[3], ki);
  const uint32_t mine = ((1u << U) - 1u) << (lane / U * U);
  if (u == 0 && (nan_lanes & mine)) k0 = (k0 & ~0xffu) | 0x7fu;
  if (on) {
    *reinterpret_cast<uint32_t*>(k_row + ld.a) = k0;
    *reinterpret_cast<uint32_t*>(k_row + ld.b) = quant4(kx[4], kx[5], kx[6], kx[7], ki);
    *reinterpret_cast<uint32_t*>(v_row + ld.a) = quant4(vx[0], vx[1], vx[2], vx[3], vi);
    *reinterpret_cast<uint32_t*>(v_row + ld.b) = quant4(vx[4], vx[5], vx[6], vx[7], vi);
  }
}

// Sixteen rows of a head by one warp: all of them on their way to shared memory
// at once, and read there twice, for the maximum and for the rounding.  The
// loops over passes stay rolled: unrolled, the instruction fetch bound the
// kernel.
template <int D>
struct Stage16 {
  static constexpr int ROW = D * 2, BYTES = 2 * 16 * ROW;   // keys, then values
};

// Whether a page's angles are kept in shared memory for the heads that use them:
// up to 8 KB, which costs no block its place (61 ragged questions, pages of 16,
// half of d turned: 13.2 us from the table, 12.0 so; pages of 64, all of d turned,
// 32 KB: 165 and 181 for a document of 16384 tokens).
__host__ __device__ inline bool keep_angles(int page, int rot) {
  return rot > 0 && page * rot * 4 <= 8192;
}

// Rows [i, i + nr) of the call into slots [off, off + nr) of head h of page pg
// by the `wph` warps of a head, 16 rows each; all of the block's warps call it
// (live: this one has a head), for its one barrier.  angles: of the page's rows,
// in the table or, where they are few, in shared memory.
template <int D, int WARPS, bool INTER>
__device__ __forceinline__ void write_group(const AppendParams& p, int i, int nr, int pg,
                                            int off, int h, bool live, int part, int wph,
                                            float2 (&red)[WARPS], uint8_t* stage,
                                            const float* angles, int warp,
                                            int lane) {
  using S = Stage16<D>;
  constexpr int U = D / 8, RP = 32 / U;               // units a row, rows a pass
  const int u = lane % U, rl = lane / U;
  const LaneDims ld = lane_dims<INTER>(p, u);
  const int64_t cell = (int64_t)pg * p.L.H + h;
  uint8_t* kb = p.L.k + cell * p.L.page * D;
  uint8_t* vb = p.L.v + cell * p.L.page * D;
  const int r0 = part * 16;
  const int mine = live ? min(16, nr - r0) : 0;       // rows of this warp
  float ko = 0.f, vo = 0.f;
  if (live && off > 0) {
    ko = p.L.k_scale[cell];
    vo = p.L.v_scale[cell];
  }
  __syncwarp();                                       // the head before is out of the stage
  {
    const uint16_t* ks = p.k + (int64_t)(i + r0 + rl) * p.k_ld + (int64_t)h * D + u * 8;
    const uint16_t* vs = p.v + (int64_t)(i + r0 + rl) * p.v_ld + (int64_t)h * D + u * 8;
    uint32_t to = smem_u32(stage) + rl * S::ROW + u * 16;
#pragma unroll 2
    for (int r = rl; r < mine; r += RP) {
      cp_async16(to, ks, 16);
      cp_async16(to + 16 * S::ROW, vs, 16);
      ks += RP * p.k_ld;
      vs += RP * p.v_ld;
      to += RP * S::ROW;
    }
  }
  cp_async_wait_all();
  __syncwarp();
  const uint8_t* at_a = stage + ld.a * 2;             // the lane's groups of key row 0
  const uint8_t* at_b = stage + ld.b * 2;
  auto key = [&](int r, float (&x)[8]) {
    unpack8(*reinterpret_cast<const uint2*>(at_a + r * S::ROW),
            *reinterpret_cast<const uint2*>(at_b + r * S::ROW), x);
    if (ld.turns) {
      const float* t = angles + (r0 + r) * p.rot + u * 4;
      turn8<INTER>(*reinterpret_cast<const float4*>(t),
                   *reinterpret_cast<const float4*>(t + (p.rot >> 1)), x);
    }
  };
  auto value_bits = [&](int r, uint2& a, uint2& b) {
    a = *reinterpret_cast<const uint2*>(at_a + (16 + r) * S::ROW);
    b = *reinterpret_cast<const uint2*>(at_b + (16 + r) * S::ROW);
  };
  float ka = 0.f;                                     // NaN once a key is
  uint32_t va2 = 0;                                   // bf16 magnitudes, as bits, two columns
#pragma unroll 2
  for (int r = rl; r < mine; r += RP) {
    float x[8];
    key(r, x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(ka) : "f"(fabsf(x[e])));
    uint2 a, b;
    value_bits(r, a, b);
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      asm("max.u16x2 %0, %0, %1;" : "+r"(va2) : "r"(w[c] & 0x7fff7fffu));
  }
  const uint32_t vm = max(va2 & 0xffffu, va2 >> 16);
  float va = __uint_as_float(vm << 16);
  const bool bad = __any_sync(0xffffffffu, !(ka < INFINITY) || vm >= 0x7f80u);
  if (bad) {                                          // rare: the largest finite ones
    if (lane == 0) set_status(p.L.status, PP_DEV_NONFINITE);
    ka = va = 0.f;
    bool any = false;
    for (int r = rl; r < mine; r += RP) {
      float x[8];
      key(r, x);
      amax8(x, ka, any);
      uint2 a, b;
      value_bits(r, a, b);
      unpack8(a, b, x);
      amax8(x, va, any);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
    va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
  }
  // (the barrier also has every warp's look at the old scales behind it before
  // one of them is overwritten)
  if (lane == 0) red[warp] = make_float2(ka, va);
  __syncthreads();
  if (!live) return;
  for (int w = 0; w < wph; ++w) {
    const float2 y = red[warp - part + w];
    ka = fmaxf(ka, y.x);
    va = fmaxf(va, y.y);
  }
  float ks = scale_for(ka), vs = scale_for(va);
  if (off > 0) {
    if (ks > ko) requant<D>(kb, off, ko / ks, part * 32 + lane, wph * 32);
    else ks = ko;
    if (vs > vo) requant<D>(vb, off, vo / vs, part * 32 + lane, wph * 32);
    else vs = vo;
  }
  if (part == 0 && lane == 0) {
    p.L.k_scale[cell] = ks;
    p.L.v_scale[cell] = vs;
  }
  const float ki = 1.f / ks, vi = 1.f / vs;
  uint8_t* k_row = kb + (off + r0 + rl) * D;
  uint8_t* v_row = vb + (off + r0 + rl) * D;
#pragma unroll 2
  for (int q = 0; q < mine; q += RP) {
    const int r = q + rl < mine ? q + rl : 0;
    float kx[8], vx[8];
    key(r, kx);
    uint2 a, b;
    value_bits(r, a, b);
    unpack8(a, b, vx);
    put8<D>(k_row, v_row, ld, u, q + rl < mine, kx, vx, ki, vi, bad, lane);
    k_row += RP * D;
    v_row += RP * D;
  }
}

constexpr int kShortWarps = 4;

// The same without stages, for calls of many short runs (a decode step): a warp
// takes 32 / U heads side by side, U lanes each (h: the lane's), and of the run's
// rows W = 1: all, W = kShortWarps: its share, the block's warps together.
template <int D, bool INTER, int W>
__device__ __forceinline__ void write_short(const AppendParams& p, int i, int nr, int pos0, int pg,
                                            int off, int h, bool live,
                                            float2 (*red)[kShortWarps][256 / D], int warp,
                                            int lane) {
  constexpr int U = D / 8;
  const int u = lane % U, r0 = W == 1 ? 0 : warp;
  const LaneDims ld = lane_dims<INTER>(p, u);
  const int64_t cell = (int64_t)pg * p.L.H + h;
  uint8_t* kb = p.L.k + cell * p.L.page * D;
  uint8_t* vb = p.L.v + cell * p.L.page * D;
  float ko = 0.f, vo = 0.f;
  if (live && off > 0) {
    ko = p.L.k_scale[cell];
    vo = p.L.v_scale[cell];
  }
  float kx[8], vx[8], ka = 0.f, va = 0.f;
  bool bad = false;
  auto load = [&](int r) {
    const uint16_t* k = p.k + (int64_t)(i + r) * p.k_ld + (int64_t)h * D;
    const uint16_t* v = p.v + (int64_t)(i + r) * p.v_ld + (int64_t)h * D;
    unpack8(__ldg(reinterpret_cast<const uint2*>(k + ld.a)),
            __ldg(reinterpret_cast<const uint2*>(k + ld.b)), kx);
    unpack8(__ldg(reinterpret_cast<const uint2*>(v + ld.a)),
            __ldg(reinterpret_cast<const uint2*>(v + ld.b)), vx);
    if (ld.turns) turn8_at<INTER>(p, pos0 + r, u, kx);
  };
  for (int r = r0; r < nr; r += W) {
    load(r);
    amax8(kx, ka, bad);
    amax8(vx, va, bad);
  }
#pragma unroll
  for (int o = U / 2; o > 0; o >>= 1) {
    ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
    va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
  }
  if constexpr (W > 1) {
    if (u == 0) (*red)[warp][lane / U] = make_float2(ka, va);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 y = (*red)[w][lane / U];
      ka = fmaxf(ka, y.x);
      va = fmaxf(va, y.y);
    }
  }
  bad = __any_sync(0xffffffffu, bad && live);
  if (bad && lane == 0) set_status(p.L.status, PP_DEV_NONFINITE);
  float ks = scale_for(ka), vs = scale_for(va);
  if (live && off > 0) {
    const int t = r0 * U + u;
    if (ks > ko) requant<D>(kb, off, ko / ks, t, W * U);
    else ks = ko;
    if (vs > vo) requant<D>(vb, off, vo / vs, t, W * U);
    else vs = vo;
  }
  __syncwarp();
  if (live && u == 0 && r0 == 0) {
    p.L.k_scale[cell] = ks;
    p.L.v_scale[cell] = vs;
  }
  const float ki = 1.f / ks, vi = 1.f / vs;
  for (int r = r0; r < nr; r += W) {
    if (nr > 1) load(r);
    put8<D>(kb + (off + r) * D, vb + (off + r) * D, ld, u, live, kx, vx, ki, vi, bad, lane);
  }
}

// Of the rows before i: how many are of stream s (joined to cnt), and the last
// that is not (joined to last); 16 bytes of ids a thread at a time, thread t of nt.
__device__ __forceinline__ void scan_ids(const int16_t* sid, int i, int s, int t, int nt, int& cnt,
                                         int& last) {
  auto one = [&](int j, int id) {
    const bool same = id == s;
    cnt += same ? 1 : 0;
    last = same ? last : max(last, j);
  };
  const int lead = min(i, (int)((16 - (reinterpret_cast<uintptr_t>(sid) & 15)) & 15) / 2);
  const int vecs = (i - lead) / 8;
  for (int j = t; j < lead; j += nt) one(j, sid[j]);
#pragma unroll 4
  for (int v = t; v < vecs; v += nt) {
    const int4 w = __ldg(reinterpret_cast<const int4*>(sid + lead) + v);
    const int a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      one(lead + v * 8 + 2 * c, (int)(int16_t)(a[c] & 0xffff));
      one(lead + v * 8 + 2 * c + 1, a[c] >> 16);
    }
  }
  for (int j = lead + vecs * 8 + t; j < i; j += nt) one(j, sid[j]);
}

// What a warp knows of its block's window of rows, a lane each.
struct Window {
  int s, ps;             // the lane's row: stream and position
  uint32_t leaders;      // rows that are the first of their run in a page
};
__device__ __forceinline__ Window look(const AppendParams& p, int w0, int w1, bool tell, int lane) {
  const int row = w0 + lane;
  Window w{-1, -1, 0};
  int err = 0;
  bool lead = false;
  if (row < w1) {
    w.s = p.sid[row];
    w.ps = p.pos[row];
  }
  // the row before: a lane's neighbour, the window's first row's from memory
  int s_b = -1, ps_b = -1;
  if (lane == 0 && w0 > 0) {
    s_b = p.sid[w0 - 1];
    ps_b = p.pos[w0 - 1];
  }
  const int s_n = __shfl_up_sync(0xffffffffu, w.s, 1), ps_n = __shfl_up_sync(0xffffffffu, w.ps, 1);
  if (lane > 0) {
    s_b = s_n;
    ps_b = ps_n;
  }
  if (row < w1) {
    if (w.s > p.L.P_max) {
      err = PP_DEV_BAD_STREAM;
    } else if (w.s >= 0) {
      const int slot = w.s == 0 ? w.ps : w.ps - p.L.pos0;
      if (w.ps < 0 || slot < 0)
        err = w.s == 0 ? PP_DEV_DOC_OUT_OF_RANGE : PP_DEV_BAD_POSITION;
      else    // a row that follows its neighbour within a page is not a leader
        lead = row == 0 || slot % p.L.page == 0 || s_b != w.s || ps_b != w.ps - 1;
    }
  }
  if (tell && err) set_status(p.L.status, err);
  w.leaders = __ballot_sync(0xffffffffu, lead);
  return w;
}

// A leader's page and the rows of its run that fall into it, found by a warp.
struct Lead {
  int i, s, ps, off, pg, nr;
  bool fits;             // inside the table
};
__device__ __forceinline__ Lead open_lead(const AppendParams& p, int i, int s, int ps, int lane) {
  const int page = p.L.page;
  const int slot = s == 0 ? ps : ps - p.L.pos0, seg = slot / page;
  Lead x{i, s, ps, slot % page, -1, 1, seg < (s == 0 ? p.L.doc_pages : p.L.seg_pages)};
  if (x.fits)
    x.pg = page_of(s == 0 ? p.L.doc_table[seg]
                          : p.L.seg_table[(int64_t)(s - 1) * p.L.seg_pages + seg], p.L.n_pages);
  const int most = min(page - x.off, p.n - i);
  for (int r0 = 1; r0 < most; r0 += 32) {
    const int r = r0 + lane;
    const bool in = r < most && p.sid[i + r] == s && (int64_t)p.pos[i + r] == (int64_t)ps + r;
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    x.nr = r0 + (m == 0xffffffffu ? 32 : __ffs(~m) - 1);
    if (m != 0xffffffffu) break;
  }
  return x;
}

// The rows to write (none: 0) of a leader whose stream has cnt rows before it, the
// last row of another being `last`: the stream's rows must all stand next to each
// other, the leader at the position that its distance from their first asks for, and
// in the middle of a page only that first one leads.  So a page has one leader: a
// row's position names its place in the run, and a page that the run enters at slot
// 0 is entered by one row only.  (Positions between are not read: every leader would
// read all before it, 173 us instead of 165 for a document of 16384 tokens, 32 heads,
// 180 instead of 120 for 60000 tokens, 4 heads.)
__device__ __forceinline__ int rows_of(const AppendParams& p, const Lead& x, int cnt, int last,
                                       bool tell) {
  const int a = last + 1;               // first row of the run
  int err = 0, nr = x.nr;
  if (cnt != x.i - a || (int64_t)x.ps - p.pos[a] != x.i - a || (x.off > 0 && x.i > a))
    err = PP_DEV_ROW_ORDER;
  else if (!x.fits) err = x.s == 0 ? PP_DEV_DOC_OUT_OF_RANGE : PP_DEV_SEGMENT_OVERFLOW;
  else if (x.pg < 0) err = PP_DEV_BAD_PAGE;
  if (err) {
    nr = 0;
  } else if (p.rot && x.ps + nr > p.max_pos) {       // past the angle table
    err = PP_DEV_BAD_POSITION;
    nr = max(0, p.max_pos - x.ps);
  }
  if (err && tell) set_status(p.L.status, err);
  return nr;
}

// Turn the window's queries: a warp a row, four passes of heads in flight.
template <int D, int WARPS, bool INTER>
__device__ __forceinline__ void turn_queries(const AppendParams& p, int w0, int w1, int hb, int he,
                                             int warp, int lane) {
  constexpr int U = D / 8, RP = 32 / U;
  const int u = lane % U, hl = lane / U;
  const LaneDims ld = lane_dims<INTER>(p, u);
  const int row = w0 + lane;
  const int s_l = row < w1 ? p.sid[row] : -1, ps_l = row < w1 ? p.pos[row] : -1;
  for (int i = w0 + warp; i < w1; i += WARPS) {
    const int s = __shfl_sync(0xffffffffu, s_l, i - w0), ps = __shfl_sync(0xffffffffu, ps_l, i - w0);
    if (s < 0 || s > p.L.P_max || ps < 0 || (p.rot && ps >= p.max_pos)) continue;
    const uint16_t* src = p.q + (int64_t)i * p.q_ld;
    uint16_t* dst = p.q_out + (int64_t)i * p.qo_ld;
    for (int h0 = hb; h0 < he; h0 += 4 * RP) {
      uint2 a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = h0 + j * RP + hl;
        a[j] = b[j] = make_uint2(0, 0);
        if (h < he) {
          a[j] = *reinterpret_cast<const uint2*>(src + (int64_t)h * D + ld.a);
          b[j] = *reinterpret_cast<const uint2*>(src + (int64_t)h * D + ld.b);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = h0 + j * RP + hl;
        float x[8];
        unpack8(a[j], b[j], x);
        if (ld.turns) turn8_at<INTER>(p, ps, u, x);
        if (h < he) {
          *reinterpret_cast<uint2*>(dst + (int64_t)h * D + ld.a) =
              make_uint2(f2_to_bf2(x[0], x[1]), f2_to_bf2(x[2], x[3]));
          *reinterpret_cast<uint2*>(dst + (int64_t)h * D + ld.b) =
              make_uint2(f2_to_bf2(x[4], x[5]), f2_to_bf2(x[6], x[7]));
        }
      }
    }
  }
}

// WARPS: 4, or 8 for pages of 128 tokens.
template <int D, int WARPS, bool INTER>
__global__ void __launch_bounds__(WARPS * 32, 24 / WARPS) kv8_append(const AppendParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = blockIdx.x * p.win;
  const int w1 = min(p.n, w0 + p.win);
  if ((int)blockIdx.y >= p.ys) {
    const int part = blockIdx.y - p.ys, parts = gridDim.y - p.ys;
    turn_queries<D, WARPS, INTER>(p, w0, w1, p.Hq * part / parts, p.Hq * (part + 1) / parts, warp, lane);
    return;
  }
  __shared__ int red_cnt[WARPS], red_last[WARPS];
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ float2 red[2][WARPS];
  const int wph = p.L.page >> 4;                    // warps a head
  const int hpp = WARPS / wph;                      // heads a pass
  const int hb = p.L.H * (int)blockIdx.y / p.ys, he = p.L.H * ((int)blockIdx.y + 1) / p.ys;
  const bool first_cta = blockIdx.y == 0 && warp == 0;
  Window w = look(p, w0, w1, first_cta, lane);      // every warp alike
  float* staged = reinterpret_cast<float*>(stage + WARPS * Stage16<D>::BYTES);
  const bool keep = keep_angles(p.L.page, p.rot);
  int buf = 0;
  while (w.leaders) {                   // the same in every warp
    if (keep) __syncthreads();          // the leader before is done with its angles
    const int l = __ffs(w.leaders) - 1;
    w.leaders &= w.leaders - 1;
    const Lead x = open_lead(p, w0 + l, __shfl_sync(0xffffffffu, w.s, l),
                             __shfl_sync(0xffffffffu, w.ps, l), lane);
    const float* angles = p.cos_sin + (int64_t)x.ps * p.rot;  // the rows' lie in a row
    if (keep) {
      const int n16 = min(x.nr, max(0, p.max_pos - x.ps)) * (p.rot / 4);
      for (int c = threadIdx.x; c < n16; c += blockDim.x)
        cp_async16(smem_u32(staged + c * 4), angles + c * 4, 16);
      angles = staged;
    }
    int cnt = 0, last = -1;
    scan_ids(p.sid, x.i, x.s, threadIdx.x, WARPS * 32, cnt, last);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
      last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    }
    __syncthreads();
    if (lane == 0) {
      red_cnt[warp] = cnt;
      red_last[warp] = last;
    }
    __syncthreads();
    cnt = 0;
    last = -1;
#pragma unroll
    for (int v = 0; v < WARPS; ++v) {
      cnt += red_cnt[v];
      last = max(last, red_last[v]);
    }
    const int nr = rows_of(p, x, cnt, last, first_cta && lane == 0);
    if (keep) {
      cp_async_wait_all();
      __syncthreads();
    }
    if (nr == 0) continue;
    for (int h0 = hb; h0 < he; h0 += hpp) {
      const int h = h0 + warp / wph;
      write_group<D, WARPS, INTER>(p, x.i, nr, x.pg, x.off, h, h < he, warp % wph, wph, red[buf],
                                   stage + warp * Stage16<D>::BYTES, angles, warp, lane);
      buf ^= 1;
    }
  }
}

// For calls of many short runs: a warp takes a leader of the window by itself, and
// the block's warps together the runs of more than kAlone rows.  (All rows of a run
// by the warp that has its heads: a step of 256 rows, 32 heads 7.1 us, so 7.8; but a
// question of 250 rows 60 and 22, a document's 1000 133 and 46.)
constexpr int kAlone = 2;
template <int D, bool INTER>
__global__ void __launch_bounds__(kShortWarps * 32, 32 / kShortWarps)
    kv8_append_short(const AppendParams p) {
  constexpr int HW = 256 / D;           // heads a warp takes side by side
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = blockIdx.x * p.win;
  const int w1 = min(p.n, w0 + p.win);
  if ((int)blockIdx.y >= p.ys) {
    const int part = blockIdx.y - p.ys, parts = gridDim.y - p.ys;
    turn_queries<D, kShortWarps, INTER>(p, w0, w1, p.Hq * part / parts, p.Hq * (part + 1) / parts,
                                        warp, lane);
    return;
  }
  __shared__ int rows[32];              // of a leader, where the block shares it
  __shared__ int page_at[32], off_at[32];
  __shared__ float2 red[2][kShortWarps][HW];
  const int hb = p.L.H * (int)blockIdx.y / p.ys, he = p.L.H * ((int)blockIdx.y + 1) / p.ys;
  const Window w = look(p, w0, w1, blockIdx.y == 0 && warp == 0, lane);
  const int hl = lane / (D / 8);
  auto skip = [](uint32_t m, int k) {   // all but its first k leaders
#pragma unroll
    for (int z = 0; z < kShortWarps; ++z) m = z < k ? m & (m - 1) : m;
    return m;
  };
  for (uint32_t m = skip(w.leaders, warp); m; m = skip(m, kShortWarps)) {
    const int l = __ffs(m) - 1;
    const Lead x = open_lead(p, w0 + l, __shfl_sync(0xffffffffu, w.s, l),
                             __shfl_sync(0xffffffffu, w.ps, l), lane);
    int cnt = 0, last = -1;
    scan_ids(p.sid, x.i, x.s, lane, 32, cnt, last);
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    last = __reduce_max_sync(0xffffffffu, last);
    const int nr = rows_of(p, x, cnt, last, blockIdx.y == 0 && lane == 0);
    if (lane == 0) rows[l] = nr > kAlone ? nr : 0;
    if (nr > kAlone && lane == 0) {
      page_at[l] = x.pg;
      off_at[l] = x.off;
    }
    if (nr == 0 || nr > kAlone) continue;
    for (int h0 = hb; h0 < he; h0 += HW) {
      const int h = h0 + hl;
      write_short<D, INTER, 1>(p, x.i, nr, x.ps, x.pg, x.off, h < he ? h : hb, h < he, nullptr, warp,
                               lane);
    }
  }
  if (w.leaders == 0) return;           // (the same in every warp)
  __syncthreads();
  int buf = 0;
  for (uint32_t m = w.leaders; m; m &= m - 1) {
    const int l = __ffs(m) - 1, nr = rows[l];
    if (nr == 0) continue;
    const int ps = __shfl_sync(0xffffffffu, w.ps, l);
    for (int h0 = hb; h0 < he; h0 += HW) {
      const int h = h0 + hl;
      write_short<D, INTER, kShortWarps>(p, w0 + l, nr, ps, page_at[l], off_at[l], h < he ? h : hb,
                                         h < he, &red[buf], warp, lane);
      buf ^= 1;
    }
  }
}

__global__ void kv8_clear_status(int32_t* status) { *status = 0; }

template <int D, int WARPS, bool INTER>
cudaError_t start_long(const AppendParams& p, dim3 grid, cudaStream_t st) {
  // the stages, and the angles of a page's rows
  constexpr int MOST = WARPS * Stage16<D>::BYTES + 8192;
  const int smem = WARPS * Stage16<D>::BYTES +
                   (keep_angles(p.L.page, p.rot) ? p.L.page * p.rot * 4 : 0);
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    e = cudaFuncSetAttribute(kv8_append<D, WARPS, INTER>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  kv8_append<D, WARPS, INTER><<<grid, WARPS * 32, smem, st>>>(p);
  return cudaGetLastError();
}
template <int D, bool INTER>
cudaError_t start(const AppendParams& p, bool brief, int warps, dim3 grid, cudaStream_t st) {
  if (brief) {
    kv8_append_short<D, INTER><<<grid, kShortWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
  }
  return warps == 8 ? start_long<D, 8, INTER>(p, grid, st) : start_long<D, 4, INTER>(p, grid, st);
}

}  // namespace

cudaError_t launch_kv8_reset(const pp_kv8_layer& L, cudaStream_t st) {
  kv8_clear_status<<<1, 1, 0, st>>>(L.status);
  return cudaGetLastError();
}

cudaError_t launch_kv8_append(const pp_kv8_layer& L, const pp_kv8_append_args& a, int num_sms,
                              cudaStream_t st) {
  AppendParams p{};
  const int n = a.n, Hq = a.q ? a.Hq : 0;
  p.L = L;
  p.k = a.k; p.v = a.v; p.q = a.q; p.q_out = a.q_out;
  p.k_ld = a.k_ld; p.v_ld = a.v_ld; p.q_ld = a.q_ld; p.qo_ld = a.q_out_ld;
  p.Hq = Hq;
  p.n = n;
  p.sid = a.sid; p.pos = a.pos;
  if (a.rope) {
    p.cos_sin = a.rope->cos_sin;
    p.rot = a.rope->dim;
    p.interleaved = a.rope->interleaved;
    p.max_pos = a.rope->max_pos;
  }
  // A CTA looks after a window of rows for a share of the heads.  Windows are
  // long (most rows of a long run are no leaders, and a CTA that only finds
  // that out costs a launch slot) and shares small, as far as the grid stays
  // between a few CTAs an SM and about 64.
  // A stream has one run a call, so more rows than streams means long runs.
  // (A decode step of 256 streams, 32 heads by the long form took 54 us, a question
  // of 250 rows 12 by it and 22 by the short one.)
  const bool brief = n <= L.P_max;
  const int warps = brief ? kShortWarps : L.page == 128 ? 8 : 4;
  const int hpp = brief ? 256 / L.d : warps / (L.page >> 4);
  const int passes = (L.H + hpp - 1) / hpp;
  p.win = brief ? kShortWarps : 1;
  const int64_t most = (brief ? 32LL : 8LL) * num_sms;   // (a short form's block is small)
  while (p.win < 32 && (int64_t)((n + p.win - 1) / p.win) * passes > most) p.win *= 2;
  const int64_t wins = (n + p.win - 1) / p.win;
  // scanning the ids before a leader is the share's fixed cost: fewer shares
  // for long calls
  p.ys = passes;
  while (p.ys > 1 && wins * (p.ys / 2) >= 8LL * num_sms) p.ys = (p.ys + 1) / 2;
  const int qh = p.win > 4 ? 1024 / L.d : 16;   // heads of a block that turns queries
  const int qs = (Hq + qh - 1) / qh;
  const dim3 grid((unsigned)wins, p.ys + qs);
  if (L.d == 128)
    return p.interleaved ? start<128, true>(p, brief, warps, grid, st)
                         : start<128, false>(p, brief, warps, grid, st);
  return p.interleaved ? start<64, true>(p, brief, warps, grid, st)
                       : start<64, false>(p, brief, warps, grid, st);
}

}  // namespace pp
