// Attention over the 8-bit paged cache on warp-level mma: the stream segments
// of a decode step or a question prefill, the document too where it is short,
// and the merge with the tensor-core document pass's partials.
//
//   w_t = scale q.k_t + log2-scale terms,  o = sum_t 2^(w_t - M) v_t / l
// over the visible slots t of a row's stream.  With x_t the stored key, a page's
// scales ks, vs (powers of two) and everything in the log2 domain,
//   w_t = (q.x_t) scale ks log2e + log2 vs,   M = max w_t,
//   O = sum 2^(w_t - M) y_t  (y the stored value),  l = sum 2^(w_t - M) / vs
// so the value scale costs one addition per page and key, not a product per
// value.
//
// One item = up to 8 * NT (query row, query head) pairs that share a key head;
// grouped query heads of a row stand together.  The products are taken
// transposed, S^T = K Q^T and O^T = V^T P^T, so the 16-wide mma dimension is
// the keys' and the values', and the 8-wide one the few rows.  A lane reads a
// key's contiguous 32 bytes (values: 16 bytes of four keys); which dims and
// keys an mma index stands for is free as long as both operands agree, so no
// value is shuffled.  e4m3 -> f16 is exact; queries are scaled by a power of
// two into f16's range; P^T goes from the accumulators to the operand by a
// transposing move.
//
// A warp brings 16 keys (K and V, 4 KB) at a time into its own ring in shared
// memory with 16-byte asynchronous copies, two chunks ahead; what bounds the
// pass is latency, so 16 (12 with two tiles of rows) warps share an SM.  WAYS
// warps share an item, each a contiguous range of its chunks; the partials meet
// in shared memory (over the rings), where each row's (m, l, O) are joined with
// the document pass's: the lanes take the partials' maxima and sums, the warp
// then adds the partials' rows with their weights known.
#include <atomic>
#include <type_traits>

#include "kv8.cuh"
#include "internal.h"
#include "warp_mma.cuh"

namespace pp {
namespace {

struct Attn8Params {
  pp_kv8_layer L;
  const uint16_t* q;
  int64_t q_ld;
  int Hq, g, hg, gt, rt;   // query heads, per key head, per item, items per key head's group, rows per item
  int rows, n_items, row_groups;
  const int16_t* q_sid;
  const int32_t* q_pos;
  int doc_len;             // document keys read here (0: none, or left to the document pass)
  float sl2;               // scale * log2e
  int ways, base;          // warps per item, and of an item of few chunks
  int lper;                // log2 of the 16-key chunks per page
  int has_doc;             // document partials to merge
  int plan32;              // the plan's divisions fit 32 bits
  SplitPlan plan;
  const float* doc_o;
  const float* doc_ml;
  uint16_t* o;
  float* lse;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 f16 matrix across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// One warp's running state over an item's rows: row n of tile t is held by the
// lanes with lane % 4 == n / 2 (n = 2c, 2c + 1).
template <int D, int NT>
struct State {
  float m[NT][2];          // running maximum of w (uniform over a row's lanes)
  float l[NT][2];          // this lane's part of the sum
  float o[NT][D / 16][4];  // O^T: [tile][dim pair j][2 rows x 2 dims]
};

// ---- the warp's ring: a stage holds 16 keys' rows, then their values'
template <int D>
struct Ring {
  static constexpr int ST = D == 128 ? 3 : 4;         // stages
  static constexpr int HALF = 16 * D, STAGE = 2 * HALF;
  static constexpr int BYTES = ST * STAGE;
};

// Byte offset of 16-byte unit u of row `row`; units are XOR-ed with the row (two
// rows of 64 bytes to a line) so that eight lanes' reads meet 32 banks.
template <int D>
__device__ __forceinline__ uint32_t unit_off(int row, int u) {
  if constexpr (D == 128) return (uint32_t)(row * 128 + ((u ^ (row & 7)) << 4));
  const int line = row >> 1;
  return (uint32_t)(line * 128 + ((((row & 1) * 4 + u) ^ ((line & 3) * 2)) << 4));
}

template <int D>
__device__ __forceinline__ void fetch_chunk(uint32_t stage, const uint8_t* kb, const uint8_t* vb,
                                            int lane) {
  constexpr int U = D / 16;
#pragma unroll
  for (int i = 0; i < 16 * U / 32; ++i) {
    const int x = lane + 32 * i;
    const uint32_t at = stage + unit_off<D>(x / U, x % U);
    cp_async16(at, kb + x * 16, 16);
    cp_async16(at + Ring<D>::HALF, vb + x * 16, 16);
  }
}

// Keys t0 .. t0 + 15; lim[t][e]: last visible slot of row 2c + e of tile t.
// t_max: the largest of all rows' lims; a key past it holds whatever the page
// held before, so its values are taken as 0 (0 * NaN would spoil the sum).
template <int D, int NT>
__device__ __forceinline__ void chunk_step(State<D, NT>& st, const uint32_t (&qf)[NT][D / 8],
                                           const uint8_t* stage, int t0, const int (&lim)[NT][2],
                                           int t_max, int t_min, const float (&qs)[NT][2],
                                           float ks, float vs, int r, int c) {
  float s[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
  uint32_t kx[2][D / 16];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      *reinterpret_cast<uint4*>(&kx[a][4 * i]) = *reinterpret_cast<const uint4*>(
          stage + unit_off<D>(r + 8 * a, c * (D / 64) + i));
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t a0 = e4m3x2_to_h2(kx[0][kk]), a2 = e4m3x2_hi_to_h2(kx[0][kk]);
    const uint32_t a1 = e4m3x2_to_h2(kx[1][kk]), a3 = e4m3x2_hi_to_h2(kx[1][kk]);
#pragma unroll
    for (int t = 0; t < NT; ++t) mma_f16(s[t], a0, a1, a2, a3, qf[t][2 * kk], qf[t][2 * kk + 1]);
  }
  const float lv = (float)((int)(__float_as_uint(vs) >> 23) - 127);   // log2 vs
  const float rvs = 1.f / vs;
  bool up = false;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = qs[t][e] * ks;
      s[t][e] = fmaf(s[t][e], a, lv);
      s[t][2 + e] = fmaf(s[t][2 + e], a, lv);
      if (t0 + 15 > t_min) {
        if (t0 + r > lim[t][e]) s[t][e] = -INFINITY;
        if (t0 + r + 8 > lim[t][e]) s[t][2 + e] = -INFINITY;
      }
      // (a NaN score counts as a new maximum: its row comes out NaN)
      up |= !(s[t][e] <= st.m[t][e]) || !(s[t][2 + e] <= st.m[t][e]);
    }
  if (__any_sync(0xffffffffu, up)) {      // some row's maximum rises: move all to their new ones
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x0 = s[t][e] != s[t][e] ? INFINITY : s[t][e];
        const float x1 = s[t][2 + e] != s[t][2 + e] ? INFINITY : s[t][2 + e];
        float x = fmaxf(x0, x1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        const float m = fmaxf(st.m[t][e], x);
        const float f = m == -INFINITY ? 1.f : ex2_mufu(st.m[t][e] - m);
        st.m[t][e] = m;
        st.l[t][e] *= f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          st.o[t][j][e] *= f;
          st.o[t][j][2 + e] *= f;
        }
      }
  }
  uint32_t pb[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float pr[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float m = st.m[t][e] == -INFINITY ? 0.f : st.m[t][e];
      pr[e] = ex2_mufu(s[t][e] - m);
      pr[2 + e] = ex2_mufu(s[t][2 + e] - m);
      st.l[t][e] = fmaf(pr[e] + pr[2 + e], rvs, st.l[t][e]);
    }
    // P to f16: 2^-11 of its value, against e4m3's 2^-4 of the values it weighs
    pb[t][0] = transpose8(f2_to_h2(pr[0], pr[1]));
    pb[t][1] = transpose8(f2_to_h2(pr[2], pr[3]));
  }
  uint32_t vx[4][D / 32];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int row = 2 * c + (a & 1) + 8 * (a >> 1);
    const uint8_t* at = stage + Ring<D>::HALF;
    if constexpr (D == 128)
      *reinterpret_cast<uint4*>(&vx[a][0]) =
          *reinterpret_cast<const uint4*>(at + unit_off<D>(row, r));
    else
      *reinterpret_cast<uint2*>(&vx[a][0]) =
          *reinterpret_cast<const uint2*>(at + unit_off<D>(row, r >> 1) + (r & 1) * 8);
  }
  if (t0 + 15 > t_max) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (t0 + 2 * c + (a & 1) + 8 * (a >> 1) > t_max)
#pragma unroll
        for (int w = 0; w < D / 32; ++w) vx[a][w] = 0u;
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {      // 4 bytes of each value row: dims 4w .. 4w + 3 of the lane's
    // two keys' bytes interleaved, then to f16: dims 4w + (0, 1 | 2, 3)
    const uint32_t ka0 = __byte_perm(vx[0][w], vx[1][w], 0x5140), ka1 = __byte_perm(vx[0][w], vx[1][w], 0x7362);
    const uint32_t kb0 = __byte_perm(vx[2][w], vx[3][w], 0x5140), kb1 = __byte_perm(vx[2][w], vx[3][w], 0x7362);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t ka = i ? ka1 : ka0, kb = i ? kb1 : kb0;
      const uint32_t a0 = e4m3x2_to_h2(ka), a1 = e4m3x2_hi_to_h2(ka);
      const uint32_t a2 = e4m3x2_to_h2(kb), a3 = e4m3x2_hi_to_h2(kb);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_f16(st.o[t][2 * w + i], a0, a1, a2, a3, pb[t][0], pb[t][1]);
    }
  }
}

// Chunks [c0, c1) of one token sequence (page table `tab`): 32 table entries
// and scales are fetched at a time.
template <int D, int NT>
__device__ __forceinline__ void scan(State<D, NT>& st, const uint32_t (&qf)[NT][D / 8],
                                     const Attn8Params& p, const int32_t* tab, int h, int c0,
                                     int c1, const int (&lim)[NT][2], int t_max, int t_min,
                                     const float (&qs)[NT][2], uint8_t* ring, int lane) {
  constexpr int ST = Ring<D>::ST;
  const uint32_t ring_u = smem_u32(ring);
  const int lper = p.lper, per = 1 << lper;   // chunks per page: 1, 2, 4, 8
  for (int b = c0; b < c1; b += 32) {
    const int n = min(32, c1 - b);
    int pg = -1;
    float ks = 1.f, vs = 1.f;
    if (lane < n) {
      pg = page_of(tab[(b + lane) >> lper], p.L.n_pages);
      if (pg < 0) set_status(p.L.status, PP_DEV_BAD_PAGE);
    }
    auto fetch = [&](int j) {
      const int pgj = __shfl_sync(0xffffffffu, pg, j);
      if (pgj >= 0) {
        const int64_t at =
            (((int64_t)pgj * p.L.H + h) * p.L.page + ((b + j) & (per - 1)) * 16) * D;
        fetch_chunk<D>(ring_u + (j % ST) * Ring<D>::STAGE, p.L.k + at, p.L.v + at, lane);
      }
    };
#pragma unroll
    for (int j = 0; j < ST - 1; ++j) {
      if (j < n) fetch(j);
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    if (pg >= 0) {
      ks = p.L.k_scale[(int64_t)pg * p.L.H + h];
      vs = p.L.v_scale[(int64_t)pg * p.L.H + h];
    }
    for (int j = 0; j < n; ++j) {
      if (j + ST - 1 < n) fetch(j + ST - 1);
      asm volatile("cp.async.commit_group;\ncp.async.wait_group %0;\n" ::"n"(ST - 1) : "memory");
      __syncwarp();
      const float ksj = __shfl_sync(0xffffffffu, ks, j), vsj = __shfl_sync(0xffffffffu, vs, j);
      if (__shfl_sync(0xffffffffu, pg, j) >= 0)
        chunk_step<D, NT>(st, qf, ring + (j % ST) * Ring<D>::STAGE, (b + j) * 16, lim, t_max, t_min,
                          qs, ksj, vsj, lane >> 2, lane & 3);
      __syncwarp();
    }
  }
}

// A slice of chunks: part `w` of `ways` of the sequence's [0, n).
__device__ __forceinline__ void part_of(int n, int w, int ways, int& c0, int& c1) {
  c0 = (int)((int64_t)n * w / ways);
  c1 = (int)((int64_t)n * (w + 1) / ways);
}

constexpr int kMaxWays = 16;   // warps of a CTA, and of an item, at most
// An item of more chunks than this is cut where it would be one warp's.
constexpr int kShareChunks = 16;

// A warp's shared memory: its ring, and over it, when the keys are done, its
// partial result: (m, l) of its rows, then O, rows of D + 4 floats.
template <int D, int NT>
struct Smem8 {
  static constexpr int ROWS = 8 * NT, LD = D + 4;
  static constexpr int PART = ROWS * (LD + 2) * 4;
  static constexpr int WARP = PART > Ring<D>::BYTES ? (PART + 127) / 128 * 128 : Ring<D>::BYTES;
};

// Partial j of a row's document partials: slot of the row's (m, l) and O.
struct DocRow {
  int64_t slot;   // of the first
  int n;          // partials
  int two;        // a row group of one M tile: two a chunk, 128 rows apart
  __device__ __forceinline__ int64_t at(int j) const {
    return two ? slot + (int64_t)(j >> 1) * kGroupRows + (j & 1) * 128
               : slot + (int64_t)j * kGroupRows;
  }
};

// CTA of the document pass that owns step t of its plan (plan_cta_of, in 32 bits
// where they hold: a 64-bit division is some 150 instructions).
__device__ __forceinline__ int doc_cta(const Attn8Params& p, int64_t t) {
  return p.plan32 ? (int)(((uint32_t)(t + 1) * (uint32_t)p.plan.C - 1u) / (uint32_t)p.plan.W)
                  : plan_cta_of(p.plan, t);
}
// Where the document partials of (query row `row`, query head kvh * g + hq) are.
__device__ __forceinline__ DocRow doc_row(const Attn8Params& p, int row, int kvh, int hq) {
  const int pair = row * p.g + hq;                    // (the host keeps rows * Hq in 31 bits)
  const int u = kvh * p.plan.G + pair / kGroupRows;
  const int64_t ub = (int64_t)u * p.plan.T;
  DocRow d;
  d.two = p.rows * p.g - pair / kGroupRows * kGroupRows <= 128;
  d.n = (doc_cta(p, ub + p.plan.T - 1) - doc_cta(p, ub + kKv8Lead) + 1) << d.two;
  d.slot = (int64_t)u * p.plan.max_chunks * kGroupRows + pair % kGroupRows;
  return d;
}

// A lane's share of row n = 2c + a of tile t of a partial: dims (D/8) r ..
// (Partials are read by plain loads: the document pass may still write them while
// this kernel runs, and only a plain load stays behind griddepcontrol.wait.)
template <int D>
__device__ __forceinline__ void load_part(float (&x)[D / 8], const float* row, int r) {
#pragma unroll
  for (int i = 0; i < D / 8; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(row + r * (D / 8) + i);
    x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
  }
}

// The warps that share an item make a block: with four items of different
// lengths to a block the shorter ones' places stayed empty.
template <int D, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, (NT == 1 ? 16 : 12) / WARPS)
    kv8_attn(const Attn8Params p) {
  using M = Smem8<D, NT>;
  constexpr int LD = M::LD;
  extern __shared__ __align__(128) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  // ---- the warp's item: place x among those of rows rt * rg ..
  const int xs = p.L.H * p.gt;
  int ways = WARPS, rg, x;
  bool live = true;
  if (WARPS == 1 || p.base == WARPS) {
    rg = (int)blockIdx.x / xs;
    x = (int)blockIdx.x - rg * xs;
  } else {
    // The tables have room for long segments and these rows' may be short, which the
    // host does not know: then the first of a few blocks of the rows takes their
    // items, `base` warps each, and the others, which stand behind all first ones,
    // end.  (64 streams of 17..80 tokens, 32 heads, room for 1024 more 23.3 us, cut all
    // the same 33.7, in tables without room 22.5; segments of 1024 tokens pay 2 % for
    // the question, 99.7 and 97.7.)
    const int per = WARPS / p.base, groups = (xs + per - 1) / per;
    const int leaders = p.row_groups * groups;
    const bool leads = (int)blockIdx.x < leaders;
    if (leads) {
      rg = (int)blockIdx.x / groups;
      x = ((int)blockIdx.x - rg * groups) * per;
    } else {
      const int b = (int)blockIdx.x - leaders, f = xs - groups;
      rg = b / f;
      x = (b - rg * f) / (per - 1) * per + 1 + (b - rg * f) % (per - 1);
    }
    const int row = rg * p.rt + lane;
    int seg = 0;                           // 16-key chunks of the lane's row
    if (lane < p.rt && row < p.rows && p.q_pos[row] >= p.L.pos0 &&
        stream_query(p.q_sid[row], p.L.P_max))
      seg = min((p.q_pos[row] - p.L.pos0) >> 4, p.L.seg_pages * p.L.page / 16 - 1) + 1;
    seg = __reduce_max_sync(0xffffffffu, seg);
    if (seg + ((p.doc_len + 15) >> 4) <= kShareChunks * p.base) {
      if (!leads) return;
      ways = p.base;
      x += warp / ways;
      live = x < xs;
    }
  }
  const int way = warp & (ways - 1);
  uint8_t* ring = sm + warp * M::WARP;
  float* my_ml = reinterpret_cast<float*>(ring);
  float* my_o = my_ml + 2 * M::ROWS;
  int r0 = 0, kvh = 0, hb = 0, nh = 1, nrow = 0;
  if (live) {
    r0 = rg * p.rt;
    kvh = x / p.gt;
    hb = (x % p.gt) * p.hg;               // first query head inside the group
    nh = min(p.hg, p.g - hb);
    nrow = min(p.rt, p.rows - r0);
    const int n_pairs = nrow * nh;
    // ---- what the item starts from, all on its way at once: lane i's row, the
    // queries' bits, the document partials of rows that a warp has to itself
    int sid_l = -1, ps_l = -1;
    if (lane < nrow) {
      sid_l = p.q_sid[r0 + lane];
      ps_l = p.q_pos[r0 + lane];
    }
    uint32_t w2[NT][D / 8];                // bf16 pairs of row n = r of tile t
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n = t * 8 + r;
#pragma unroll
      for (int e = 0; e < D / 8; ++e) w2[t][e] = 0u;
      if (n < n_pairs) {
        const uint16_t* src = p.q + (int64_t)(r0 + n / nh) * p.q_ld +
                              (int64_t)(kvh * p.g + hb + n % nh) * D + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          *reinterpret_cast<uint4*>(&w2[t][4 * i]) = *reinterpret_cast<const uint4*>(src + 8 * i);
      }
    }
    State<D, NT> st;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        st.m[t][a] = -INFINITY;
        st.l[t][a] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) st.o[t][j][a] = st.o[t][j][2 + a] = 0.f;
      }
    DocRow dr2[NT][2];
    if (NT > 1 && p.has_doc && ways == 1) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      DocRow d{0, 0, 0};                   // of pair `lane`
      const int sid_p = __shfl_sync(0xffffffffu, sid_l, lane < n_pairs ? lane / nh : 0);
      if (lane < n_pairs && stream_query(sid_p, p.L.P_max))
        d = doc_row(p, r0 + lane / nh, kvh, hb + lane % nh);
      float2 ml[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int n2 = t * 8 + 2 * c + a;
          dr2[t][a].slot = __shfl_sync(0xffffffffu, d.slot, n2);
          dr2[t][a].n = __shfl_sync(0xffffffffu, d.n, n2);
          dr2[t][a].two = __shfl_sync(0xffffffffu, d.two, n2);
          ml[t][a] = make_float2(-INFINITY, 0.f);
          if (dr2[t][a].n == 0) continue;
          ml[t][a] = reinterpret_cast<const float2*>(p.doc_ml)[dr2[t][a].slot];
          float x[D / 8];
          load_part<D>(x, p.doc_o + dr2[t][a].slot * D, r);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            st.o[t][j][a] = x[2 * j];
            st.o[t][j][2 + a] = x[2 * j + 1];
          }
        }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          st.m[t][a] = ml[t][a].x;
          st.l[t][a] = r == 0 ? ml[t][a].y : 0.f;
          if (ml[t][a].x == -INFINITY) {   // saw no key: its O may hold anything
            st.l[t][a] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) st.o[t][j][a] = st.o[t][j][2 + a] = 0.f;
          }
        }
    }
    // ---- queries: B operand of S^T, scaled into f16
    uint32_t qf[NT][D / 8];
    float qs[NT][2];
    int lim[NT][2], sidr[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t am2 = 0;                    // largest magnitudes, as bits
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        asm("max.u16x2 %0, %0, %1;" : "+r"(am2) : "r"(w2[t][i] & 0x7fff7fffu));
      uint32_t am = max(am2 & 0xffffu, am2 >> 16);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      // 2^e with the row's largest value / 2^e in [2^13, 2^14): bf16's 8 bits are
      // exact in f16 down to 2^-30 of it; a row with a NaN or infinity is all NaN
      int e = (int)(am >> 7) - 127 - 13;
      e = e < -60 ? -60 : e;
      const float inv = am >= 0x7f80u ? __int_as_float(0x7fffffff)
                                      : __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 f = bf2_to_f2(w2[t][i]);
        qf[t][i] = f2_to_h2(f.x * inv, f.y * inv);
      }
      const float qsc = __uint_as_float((uint32_t)(e + 127) << 23) * p.sl2;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        qs[t][a] = __shfl_sync(0xffffffffu, qsc, (2 * c + a) * 4);
        const int n2 = t * 8 + 2 * c + a;
        const int at = n2 < n_pairs ? n2 / nh : 0;
        const int sd = __shfl_sync(0xffffffffu, sid_l, at), ps = __shfl_sync(0xffffffffu, ps_l, at);
        const bool on = n2 < n_pairs && stream_query(sd, p.L.P_max);
        const int cap = p.L.seg_pages * p.L.page;
        sidr[t][a] = on ? sd : 0;
        lim[t][a] = on && ps >= p.L.pos0 ? min(ps - p.L.pos0, cap - 1) : -1;
      }
    }
    // ---- document
    if (p.doc_len > 0) {
      int dl[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) dl[t][a] = sidr[t][a] ? p.doc_len - 1 : -1;
      int c0, c1;
      part_of((p.doc_len + 15) >> 4, way, ways, c0, c1);
      // rows that are no queries see nothing; t_min by the document's end
      // alone would miss them, so every chunk is masked when there are any
      bool all = true;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) all &= t * 8 + 2 * c + a >= n_pairs || sidr[t][a] != 0;
      const int t_min = __all_sync(0xffffffffu, all) ? p.doc_len - 1 : -1;
      scan<D, NT>(st, qf, p, p.L.doc_table, kvh, c0, c1, dl, p.doc_len - 1, t_min, qs, ring,
                  lane);
    }
    // ---- segments: one pass per stretch of rows of one stream
    const int before = __shfl_up_sync(0xffffffffu, sid_l, 1);
    const uint32_t starts = __ballot_sync(0xffffffffu, lane < nrow && (lane == 0 || sid_l != before));
    for (int ra = 0; ra < nrow;) {
      const int s = __shfl_sync(0xffffffffu, sid_l, ra);
      const uint32_t rest = starts >> ra >> 1;
      const int rb = rest ? ra + __ffs(rest) : nrow;
      if (s == 0 || s > p.L.P_max) {
        if (kvh == 0 && hb == 0 && way == 0 && lane == 0) set_status(p.L.status, PP_DEV_BAD_STREAM);
      } else if (s > 0) {
        int lm[NT][2], hi = -1, lo = 0x7fffffff;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const int n2 = t * 8 + 2 * c + a;
            const bool in = n2 >= ra * nh && n2 < rb * nh;
            lm[t][a] = in ? lim[t][a] : -1;
            hi = max(hi, lm[t][a]);
            // rows that hold no pair at all need no mask: nothing reads them
            if (n2 < n_pairs) lo = min(lo, lm[t][a]);
          }
#pragma unroll
        for (int o2 = 1; o2 < 4; o2 <<= 1) {
          hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o2));
          lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o2));
        }
        int c0, c1;
        part_of((hi + 16) >> 4, way, ways, c0, c1);
        scan<D, NT>(st, qf, p, p.L.seg_table + (int64_t)(s - 1) * p.L.seg_pages, kvh, c0, c1, lm,
                    hi, lo, qs, ring, lane);
      }
      ra = rb;
    }
    if (NT > 1 && ways == 1) {
      // ---- the further document partials, and out
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          float m = st.m[t][a], l = st.l[t][a];
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
          const int n2 = t * 8 + 2 * c + a;
          if (n2 >= n_pairs) continue;
          for (int k = 1; p.has_doc && k < dr2[t][a].n; ++k) {
            const int64_t sl = dr2[t][a].at(k);
            const float2 ml = reinterpret_cast<const float2*>(p.doc_ml)[sl];
            if (ml.x == -INFINITY) continue;
            float x[D / 8];
            load_part<D>(x, p.doc_o + sl * D, r);
            const float mm = fmaxf(m, ml.x);
            const float f = m == -INFINITY ? 0.f : ex2_mufu(m - mm), y = ex2_mufu(ml.x - mm);
            l = l * f + ml.y * y;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              st.o[t][j][a] = st.o[t][j][a] * f + x[2 * j] * y;
              st.o[t][j][2 + a] = st.o[t][j][2 + a] * f + x[2 * j + 1] * y;
            }
            m = mm;
          }
          const bool any = sidr[t][a] != 0 && m != -INFINITY;
          const float inv = any ? 1.f / l : 0.f;
          uint32_t w[D / 16];
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            w[j] = any ? f2_to_bf2(st.o[t][j][a] * inv, st.o[t][j][2 + a] * inv) : 0u;
          const int64_t at = (int64_t)(r0 + n2 / nh) * p.Hq + kvh * p.g + hb + n2 % nh;
#pragma unroll
          for (int j = 0; j < D / 16; j += 4)
            *reinterpret_cast<uint4*>(p.o + at * D + r * (D / 8) + 2 * j) =
                make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
          if (p.lse && r == 0) p.lse[at] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
      return;
    }
    // ---- this warp's partial to shared memory, row by row, over the ring
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float l = st.l[t][a];
#pragma unroll
        for (int o2 = 4; o2 < 32; o2 <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
        const int n2 = t * 8 + 2 * c + a;
        if (n2 >= n_pairs) continue;
        if (r == 0) {
          my_ml[2 * n2] = st.m[t][a];
          my_ml[2 * n2 + 1] = l;
        }
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)   // dims (D/8) r + 2j .. + 3
          *reinterpret_cast<float4*>(my_o + n2 * LD + r * (D / 8) + 2 * j) = make_float4(
              st.o[t][j][a], st.o[t][j][2 + a], st.o[t][j + 1][a], st.o[t][j + 1][2 + a]);
      }
  }
  if (ways > 1) __syncthreads(); else __syncwarp();
  if (!live) return;
  // (the segments did not need the document pass; its partials do)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- merge: the item's warps take its rows in turn, a lane E dims.  Lane n
  // finds where pair n's document partials are.
  constexpr int E = D / 32;
  DocRow dr{0, 0, 0};
  int q_live = 0;
  if (lane < nrow * nh) {
    const int row = r0 + lane / nh;
    q_live = stream_query(p.q_sid[row], p.L.P_max) ? 1 : 0;
    if (p.has_doc && q_live) {
      dr = doc_row(p, row, kvh, hb + lane % nh);
    }
  }
  const uint8_t* it = sm + (warp - way) * M::WARP;
  auto row_of = [&](int n) {
    DocRow d;
    d.slot = __shfl_sync(0xffffffffu, dr.slot, n);
    d.n = __shfl_sync(0xffffffffu, dr.n, n);
    d.two = __shfl_sync(0xffffffffu, dr.two, n);
    return d;
  };
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  auto doc_vec = [&](int64_t slot) {
    return reinterpret_cast<const Vec*>(p.doc_o + slot * D)[lane];
  };
  auto lane_ml = [&](const DocRow& d, int n, int j) {    // (m, l) of the row's partial j
    if (j < ways)
      return *reinterpret_cast<const float2*>(it + j * M::WARP + n * 8);
    if (j - ways < d.n)
      return reinterpret_cast<const float2*>(p.doc_ml)[d.at(j - ways)];
    return make_float2(-INFINITY, 0.f);
  };
  // the next row's maxima and first document row are on their way while one is joined
  const int n_all = nrow * nh;
  DocRow nd = row_of(way < n_all ? way : 0);
  float2 nml = make_float2(-INFINITY, 0.f);
  Vec nv{};
  if (way < n_all) {
    nml = lane_ml(nd, way, lane);
    if (nd.n) nv = doc_vec(nd.slot);
  }
  for (int n = way; n < n_all; n += ways) {
    const int row = r0 + n / nh, head = kvh * p.g + hb + n % nh;
    const DocRow d = nd;
    const float2 ml0 = nml;
    const Vec v0 = nv;
    const int n2 = n + ways;
    nd = row_of(n2 < n_all ? n2 : 0);
    if (n2 < n_all) {
      nml = lane_ml(nd, n2, lane);
      if (nd.n) nv = doc_vec(nd.slot);
    }
    const bool query = __shfl_sync(0xffffffffu, q_live, n) != 0;
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int cnt = query ? ways + d.n : 0;
    for (int b = 0; b < cnt; b += 32) {
      const float2 ml = b == 0 ? ml0 : lane_ml(d, n, b + lane);
      float mm = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
      mm = fmaxf(mm, m);
      if (mm == -INFINITY) continue;      // none of them saw a key
      const float x = m == -INFINITY ? 0.f : ex2_mufu(m - mm);
      // (of a partial that saw no key nothing is read: its O may hold anything)
      const float y = ml.x == -INFINITY ? 0.f : ex2_mufu(ml.x - mm);
      const uint32_t saw = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
      float ls = ml.x == -INFINITY ? 0.f : ml.y * y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      l = l * x + ls;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= x;
      m = mm;
      const int nb = min(32, cnt - b);
#pragma unroll 4
      for (int j = 0; j < nb; ++j) {
        const float yj = __shfl_sync(0xffffffffu, y, j);
        if (!(saw >> j & 1)) continue;
        Vec v;
        if (b + j < ways)
          v = reinterpret_cast<const Vec*>(it + j * M::WARP + M::ROWS * 8 + n * LD * 4)[lane];
        else
          v = b + j == ways ? v0 : doc_vec(d.at(b + j - ways));
        const float* f = reinterpret_cast<const float*>(&v);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(f[e], yj, acc[e]);
      }
    }
    const bool any = m != -INFINITY;
    const float inv = any ? 1.f / l : 0.f;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = any ? f2_to_bf2(acc[e] * inv, acc[e + 1] * inv) : 0u;
    uint16_t* dst = p.o + ((int64_t)row * p.Hq + head) * D + lane * E;
    if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (p.lse && lane == 0)
      p.lse[(int64_t)row * p.Hq + head] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

template <int D, int NT, int WARPS>
cudaError_t launch_as(const Attn8Params& p, cudaStream_t st) {
  constexpr int SMEM = WARPS * Smem8<D, NT>::WARP;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    e = cudaFuncSetAttribute(kv8_attn<D, NT, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  // Behind a document pass the blocks may start as its CTAs end: they read
  // the segments meanwhile and wait for it only where its partials are joined.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.n_items);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.has_doc ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv8_attn<D, NT, WARPS>, p);
}

template <int D, int NT>
cudaError_t launch(const Attn8Params& p, cudaStream_t st) {
  if constexpr (NT == 1) {
    if (p.ways > 8) return launch_as<D, NT, 16>(p, st);
    if (p.ways > 4) return launch_as<D, NT, 8>(p, st);
  }
  return p.ways > 2   ? launch_as<D, NT, 4>(p, st)
         : p.ways > 1 ? launch_as<D, NT, 2>(p, st)
                      : launch_as<D, NT, 1>(p, st);
}

}  // namespace

cudaError_t launch_kv8_attn(const pp_kv8_layer& L, const pp_kv8_attn_args& a,
                            bool one_row_per_stream, const SplitPlan& plan, bool doc_pass,
                            const Partials& part, int num_sms, cudaStream_t st) {
  Attn8Params p{};
  const int rows = a.rows;
  p.L = L;
  p.q = a.q; p.q_ld = a.q_ld;
  p.Hq = a.Hq;
  p.g = a.Hq / L.H;
  const Kv8Items it = kv8_items(rows, p.g, L.H, one_row_per_stream);
  p.hg = it.hg;
  p.gt = it.gt;
  p.rt = it.rt;
  p.rows = rows;
  const int64_t items = it.items;
  p.n_items = (int)items;
  p.q_sid = a.q_sid; p.q_pos = a.q_pos;
  p.doc_len = doc_pass ? 0 : a.doc_len;
  p.sl2 = a.scale * kLog2e;
  p.has_doc = doc_pass ? 1 : 0;
  p.plan = plan;
  p.plan32 = (plan.W + 1) * plan.C <= 0xffffffffLL;
  p.doc_o = part.doc_o; p.doc_ml = part.doc_ml;
  p.o = a.o; p.lse = a.lse;
  // Warps per item: enough to fill the GPU when items are few (they share the
  // item's merge too, however short its keys), and a long document cut so that
  // one item is not a CTA's whole tail.
  const int64_t seg_chunks = (int64_t)L.seg_pages * L.page / 16, doc_chunks = (p.doc_len + 15) / 16;
  const int most = it.most == 8 ? 8 : 4;    // (items of 16 pairs are many)
  int base = 1;
  while (base < most &&
         (items * base < 12LL * num_sms || (base < 4 && doc_chunks / base > kShareChunks)))
    base *= 2;
  // Long segments are cut too where the items are fewer than 1.5 times the GPU's
  // warps, if the kernel finds them long (the tables only tell how long they may be).
  // Measured behind 256 tokens, one warp / cut: 80 streams of 1024 tokens, 32 heads
  // 149 / 121 us, 100 167 / 146, 128 176 / 182, 256 of 300..600 159 / 200, of 1024
  // 336 / 336; a question of 2000 rows, 8 heads 161 / 106, two of 700 rows, 8 x 4 heads
  // 116 / 155.  Behind a long document one warp gains more: 128 streams of 1024 behind
  // 8192 217 / 246, 256 questions of 16..48 rows behind 12000 1486 / 1931.
  const int64_t slots = (it.most == 8 ? 16LL : 12LL) * num_sms;
  int ways = base;
  if (2 * items < 3 * slots)
    while (ways < 4 && 2 * ways <= base * (int64_t)L.H * it.gt &&
           (seg_chunks + doc_chunks) / ways > kShareChunks)
      ways *= 2;
  // (a block an SM, and keys enough to share, if the table's room is used: 4 heads,
  // segments of 1000 tokens 10.6 us so, by eight warps 10.8, of 8000 38 and 48; but
  // of 12 tokens in a table for 1024 7.7 and 6.9)
  if (base == 8 && it.most == 8 && items <= 3 * num_sms / 2 && seg_chunks + doc_chunks > 40)
    ways = base = kMaxWays;
  p.ways = ways;
  p.base = base;
  p.row_groups = (rows + it.rt - 1) / it.rt;
  p.lper = L.page == 16 ? 0 : L.page == 32 ? 1 : L.page == 64 ? 2 : 3;
  if (L.d == 128) return it.most == 8 ? launch<128, 1>(p, st) : launch<128, 2>(p, st);
  return it.most == 8 ? launch<64, 1>(p, st) : launch<64, 2>(p, st);
}

}  // namespace pp
