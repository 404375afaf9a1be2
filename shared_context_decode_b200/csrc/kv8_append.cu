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
// page's heads without any ordering between CTAs.  A run that breaks the rule
// is found by the leader's scan of the earlier stream ids and dropped.
//
// Bound: HBM (bf16 in, e4m3 out); a decode step's few kilobytes a row are
// latency.
#include "kv8.cuh"
#include "internal.h"

namespace pp {
namespace {

constexpr int kAppWarps = 4;

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
  int win;                           // rows whose leaders one CTA looks after
  int ys;                            // CTAs along y for keys and values; the rest turn queries
};

// Eight consecutive dims of a row: 16 bytes of bf16 -> floats.
__device__ __forceinline__ void load8(const uint16_t* src, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(src);
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 f = bf2_to_f2(a[c]);
    x[2 * c] = f.x;
    x[2 * c + 1] = f.y;
  }
}

// The angles' cosines and sines a lane needs for its 8 dims (unit u of the
// row): 8 pairs' when dim j turns with dim j + rot/2, 4 pairs' when 2j turns
// with 2j + 1.
__device__ __forceinline__ void load_angles(const AppendParams& p, int pos, int u, float (&cs)[8],
                                            float (&sn)[8]) {
  if (u * 8 >= p.rot) return;
  const int half = p.rot >> 1;
  const float* t = p.cos_sin + (int64_t)pos * p.rot;
  if (p.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(t + u * 4);
    const float4 s = *reinterpret_cast<const float4*>(t + half + u * 4);
    cs[0] = c.x; cs[1] = c.y; cs[2] = c.z; cs[3] = c.w;
    sn[0] = s.x; sn[1] = s.y; sn[2] = s.z; sn[3] = s.w;
  } else {
    const int j = u * 8 < half ? u * 8 : u * 8 - half;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 c = *reinterpret_cast<const float4*>(t + j + e);
      const float4 s = *reinterpret_cast<const float4*>(t + half + j + e);
      cs[e] = c.x; cs[e + 1] = c.y; cs[e + 2] = c.z; cs[e + 3] = c.w;
      sn[e] = s.x; sn[e + 1] = s.y; sn[e + 2] = s.z; sn[e + 3] = s.w;
    }
  }
}

// Rotate the lane's 8 dims.  Every product and difference is rounded by
// itself (no fused multiply-add), the result a plain fp32 evaluation of
// a cos - b sin gives, so which e4m3 value a rotated key rounds to does not
// depend on the compiler's contraction.  All lanes of the warp call it.
__device__ __forceinline__ void turn8(const AppendParams& p, int u, int lane, const float (&cs)[8],
                                      const float (&sn)[8], float (&x)[8]) {
  if (p.rot == 0) return;
  const bool in = u * 8 < p.rot;
  if (p.interleaved) {
    if (!in) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      x[2 * j] = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j]));
      x[2 * j + 1] = __fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j]));
    }
    return;
  }
  const int hu = p.rot >> 4;                       // units of a half
  const bool low = u < hu;
  const int other = in ? (low ? lane + hu : lane - hu) : lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = __shfl_sync(0xffffffffu, x[e], other);
    if (in) {
      const float c = __fmul_rn(x[e], cs[e]), s = __fmul_rn(y, sn[e]);
      x[e] = low ? __fsub_rn(c, s) : __fadd_rn(c, s);
    }
  }
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

// 8 values over a power-of-two scale -> 8 e4m3 bytes.
__device__ __forceinline__ uint2 quant8(const float (&x)[8], float inv) {
  uint2 r;
  r.x = f2_to_e4m3x2(x[0] * inv, x[1] * inv) | (f2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16);
  r.y = f2_to_e4m3x2(x[4] * inv, x[5] * inv) | (f2_to_e4m3x2(x[6] * inv, x[7] * inv) << 16);
  return r;
}

// The slots [0, n) of one head's page (n * d bytes), rounded again after its
// scale grew: x -> rn_e4m3(x * ratio), ratio = old / new < 1.
template <int D>
__device__ __forceinline__ void requant(uint8_t* base, int n, float ratio, int lane) {
  for (int c = lane; c < n * (D / 16); c += 32) {
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

// Rows [i, i + nr) of the call into slots [off, off + nr) of head h of page
// pg, by one warp: lane = (row of the pass, 8-dim unit).
template <int D>
__device__ __forceinline__ void write_group(const AppendParams& p, int i, int nr, int pos0, int pg,
                                            int off, int h, int lane) {
  constexpr int U = D / 8, RP = 32 / U;
  const int u = lane % U, rl = lane / U;
  const int64_t cell = (int64_t)pg * p.L.H + h;
  uint8_t* kb = p.L.k + cell * p.L.page * D;
  uint8_t* vb = p.L.v + cell * p.L.page * D;
  auto load = [&](int r, float (&kx)[8], float (&vx)[8]) {
    float cs[8], sn[8];
    const bool ok = r < nr;
#pragma unroll
    for (int e = 0; e < 8; ++e) kx[e] = vx[e] = cs[e] = sn[e] = 0.f;
    if (ok) {
      load8(p.k + (int64_t)(i + r) * p.k_ld + (int64_t)h * D + u * 8, kx);
      load8(p.v + (int64_t)(i + r) * p.v_ld + (int64_t)h * D + u * 8, vx);
      if (p.rot) load_angles(p, pos0 + r, u, cs, sn);
    }
    turn8(p, u, lane, cs, sn, kx);
  };
  float ka = 0.f, va = 0.f;
  bool bad = false;
  float kx[8], vx[8];
  for (int r0 = 0; r0 < nr; r0 += RP) {
    load(r0 + rl, kx, vx);
    amax8(kx, ka, bad);
    amax8(vx, va, bad);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
    va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.L.status, PP_DEV_NONFINITE);
  float ks = scale_for(ka), vs = scale_for(va);
  if (off > 0) {
    const float ko = p.L.k_scale[cell], vo = p.L.v_scale[cell];
    __syncwarp();
    if (ks > ko) requant<D>(kb, off, ko / ks, lane);
    else ks = ko;
    if (vs > vo) requant<D>(vb, off, vo / vs, lane);
    else vs = vo;
  }
  if (lane == 0) {
    p.L.k_scale[cell] = ks;
    p.L.v_scale[cell] = vs;
  }
  const float ki = 1.f / ks, vi = 1.f / vs;
  for (int r0 = 0; r0 < nr; r0 += RP) {
    if (r0 > 0 || nr > RP) load(r0 + rl, kx, vx);
    // A NaN among a row's values is kept by its key: value 0, first key
    // element NaN.  Queries that see the row come out NaN either way, and
    // queries that do not see it are not touched by 0 * NaN.
    bool vn = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool n = vx[e] != vx[e];
      vn |= n;
      vx[e] = n ? 0.f : vx[e];
    }
    const uint32_t nan_lanes = __ballot_sync(0xffffffffu, vn);
    uint2 kq = quant8(kx, ki), vq = quant8(vx, vi);
    const uint32_t mine = U == 32 ? 0xffffffffu : (((1u << U) - 1u) << (rl * U));
    if (u == 0 && (nan_lanes & mine)) kq.x = (kq.x & ~0xffu) | 0x7fu;
    if (r0 + rl < nr) {
      const int64_t at = (int64_t)(off + r0 + rl) * D + u * 8;
      *reinterpret_cast<uint2*>(kb + at) = kq;
      *reinterpret_cast<uint2*>(vb + at) = vq;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kAppWarps * 32) kv8_append(const AppendParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = blockIdx.x * p.win;
  const int w1 = min(p.n, w0 + p.win);
  if ((int)blockIdx.y >= p.ys) {
    // ---- queries: rows w0 .. w1-1, this CTA's share of the heads
    constexpr int U = D / 8, RP = 32 / U;
    const int u = lane % U, hl = lane / U;
    const int part = blockIdx.y - p.ys, parts = gridDim.y - p.ys;
    const int hb = p.Hq * part / parts, he = p.Hq * (part + 1) / parts;
    for (int i = w0; i < w1; ++i) {
      const int s = p.sid[i], ps = p.pos[i];
      if (s < 0 || s > p.L.P_max || ps < 0 || (p.rot && ps >= p.max_pos)) continue;
      float cs[8], sn[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = sn[e] = 0.f;
      if (p.rot) load_angles(p, ps, u, cs, sn);
      for (int h0 = hb + warp * RP; h0 < he; h0 += kAppWarps * RP) {
        const int h = h0 + hl;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        if (h < he) load8(p.q + (int64_t)i * p.q_ld + (int64_t)h * D + u * 8, x);
        turn8(p, u, lane, cs, sn, x);
        if (h < he) {
          uint4 r;
          r.x = f2_to_bf2(x[0], x[1]);
          r.y = f2_to_bf2(x[2], x[3]);
          r.z = f2_to_bf2(x[4], x[5]);
          r.w = f2_to_bf2(x[6], x[7]);
          *reinterpret_cast<uint4*>(p.q_out + (int64_t)i * p.qo_ld + (int64_t)h * D + u * 8) = r;
        }
      }
    }
    return;
  }
  __shared__ int red_cnt[kAppWarps], red_last[kAppWarps];
  const int page = p.L.page;
  const int hb = p.L.H * (int)blockIdx.y / p.ys, he = p.L.H * ((int)blockIdx.y + 1) / p.ys;
  for (int i = w0; i < w1; ++i) {       // every branch down to the warps' heads is CTA-uniform
    const int s = p.sid[i], ps = p.pos[i];
    if (s < 0) continue;
    const bool first_cta = blockIdx.y == 0 && threadIdx.x == 0;
    if (s > p.L.P_max) {
      if (first_cta) set_status(p.L.status, PP_DEV_BAD_STREAM);
      continue;
    }
    const int slot = s == 0 ? ps : ps - p.L.pos0;
    if (ps < 0 || slot < 0) {
      if (first_cta) set_status(p.L.status, s == 0 ? PP_DEV_DOC_OUT_OF_RANGE : PP_DEV_BAD_POSITION);
      continue;
    }
    const int off = slot % page;
    if (i > 0 && off != 0 && p.sid[i - 1] == s && p.pos[i - 1] == ps - 1) continue;  // not a leader
    // The stream's run must be its only one and its positions consecutive:
    // count the earlier rows of the stream and find the last row of another.
    int cnt = 0, last = -1;
    for (int j = threadIdx.x; j < i; j += blockDim.x) {
      const bool same = p.sid[j] == s;
      cnt += same ? 1 : 0;
      last = same ? last : j;
    }
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
    for (int w = 0; w < kAppWarps; ++w) {
      cnt += red_cnt[w];
      last = max(last, red_last[w]);
    }
    const int a = last + 1;             // first row of the run
    if (cnt != i - a || (int64_t)ps - p.pos[a] != i - a) {
      if (first_cta) set_status(p.L.status, PP_DEV_ROW_ORDER);
      continue;
    }
    const int seg = slot / page;
    if (seg >= (s == 0 ? p.L.doc_pages : p.L.seg_pages)) {
      if (first_cta)
        set_status(p.L.status, s == 0 ? PP_DEV_DOC_OUT_OF_RANGE : PP_DEV_SEGMENT_OVERFLOW);
      continue;
    }
    const int pg = page_of(s == 0 ? p.L.doc_table[seg]
                                  : p.L.seg_table[(int64_t)(s - 1) * p.L.seg_pages + seg],
                           p.L.n_pages);
    if (pg < 0) {
      if (first_cta) set_status(p.L.status, PP_DEV_BAD_PAGE);
      continue;
    }
    // rows of the run that fall into this page
    const int most = min(page - off, p.n - i);
    int nr = 1;
    for (int r0 = 1; r0 < most; r0 += 32) {
      const int r = r0 + lane;
      const bool in = r < most && p.sid[i + r] == s && (int64_t)p.pos[i + r] == (int64_t)ps + r;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      nr = r0 + (m == 0xffffffffu ? 32 : __ffs(~m) - 1);
      if (m != 0xffffffffu) break;
    }
    if (p.rot && ps + nr > p.max_pos) {   // positions past the angle table
      if (first_cta) set_status(p.L.status, PP_DEV_BAD_POSITION);
      nr = p.max_pos - ps;
      if (nr <= 0) continue;
    }
    for (int h = hb + warp; h < he; h += kAppWarps) write_group<D>(p, i, nr, ps, pg, off, h, lane);
  }
}

__global__ void kv8_clear_status(int32_t* status) { *status = 0; }

}  // namespace

cudaError_t launch_kv8_reset(const pp_kv8_layer& L, cudaStream_t st) {
  kv8_clear_status<<<1, 1, 0, st>>>(L.status);
  return cudaGetLastError();
}

cudaError_t launch_kv8_append(const pp_kv8_layer& L, const uint16_t* k, int64_t k_ld,
                              const uint16_t* v, int64_t v_ld, const uint16_t* q, int64_t q_ld,
                              int Hq, const int16_t* sid, const int32_t* pos, int n,
                              const pp_rope* rope, uint16_t* q_out, int64_t qo_ld, int num_sms,
                              cudaStream_t st) {
  AppendParams p{};
  p.L = L;
  p.k = k; p.v = v; p.q = q; p.q_out = q_out;
  p.k_ld = k_ld; p.v_ld = v_ld; p.q_ld = q_ld; p.qo_ld = qo_ld;
  p.Hq = q ? Hq : 0;
  p.n = n;
  p.sid = sid; p.pos = pos;
  if (rope) {
    p.cos_sin = rope->cos_sin;
    p.rot = rope->dim;
    p.interleaved = rope->interleaved;
    p.max_pos = rope->max_pos;
  }
  // Four warps' heads a CTA; rows by themselves while that keeps the grid
  // within a few waves, else windows of rows (most rows of a long run are not
  // leaders, and a CTA that only finds that out costs a launch slot).
  p.ys = (L.H + kAppWarps - 1) / kAppWarps;
  p.win = 1;
  while (p.win < 16 && (int64_t)((n + p.win - 1) / p.win) * p.ys > 64LL * num_sms) p.win *= 2;
  const int qs = q ? (Hq + 15) / 16 : 0;
  const dim3 grid((n + p.win - 1) / p.win, p.ys + qs);
  if (L.d == 128) kv8_append<128><<<grid, kAppWarps * 32, 0, st>>>(p);
  else kv8_append<64><<<grid, kAppWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace pp
