// Document pass over the 8-bit paged cache on the 5th-generation tensor cores.
//
// For each key head all (query row, query head) pairs that share it are
// stacked into one matrix Q; per tile of 128 document keys
//     S = Q X^T                   X the stored keys, S fp32 in TMEM
//     w = S a + log2 vs           a = query scale * page's key scale, log2 domain
//     P = 2^(w - M) as f16,  l += P / vs,  O += P Y     Y the stored values
// with M a reference for the row's maximum, so a page's value scale vs rides in
// the exponent and no value is multiplied.  M is the maximum of a run's first
// tile, and stays while a tile's sum of P stays below 2^12: then no P passes
// f16's range, and no pass over S for its maximum is needed.  A tile whose sum
// is larger raises M to its maximum, rescales O and l and is taken again (rare).
// Both products are f16 tcgen05 MMAs: e4m3 -> f16 is exact, queries are scaled
// into f16's range by a power of two a row (bf16's 8 bits fit f16's 11), and P
// keeps 2^-11 of its value.  (Products of e4m3 operands would need queries and
// probabilities as pairs of e4m3 numbers for 2^-8: the same tensor time as
// f16, and five more instructions for two probabilities in the softmax, which
// is the tighter resource.)
//
// One CTA holds two "streams": two M tiles of 128 rows over the same keys, or,
// when a row group has at most 128 rows, one M tile with even tiles on one
// stream and odd tiles on the other (two partial results).  While one stream's
// softmax runs, the tensor core works for the other; a converted tile serves
// both M tiles.  Warp roles (512 threads):
//   warp 0       loader: bulk copies of page chunks to shared memory, page
//                tables and scales (d 64: of the keys, warp 3 of the values)
//   warp 1       MMA issuer          warp 2   TMEM allocator
//   warps 4-7    e4m3 -> f16 into the MMA's 128-byte-swizzled layout
//   warps 8-15   softmax, one thread a row; queries to f16; partial results
// TMEM: O_0 | O_1 | S_0 | S_1, P over the first 64 columns of its S.
//
// Bound: the softmax warps' instruction latency.  At 256 rows, 32 heads and 16384
// keys (75 us; 134 MB, 69 GFLOP) a tile of 256 rows takes a CTA about 3450
// cycles: 1700 of exponentials on each stream, 1250 of products and hand-over
// behind them, the other stream's under both; the tensor pipe is busy for half.
//
// Every wait is bounded: on expiry the kernel sets PP_DEV_TIMEOUT, raises a
// CTA-wide abort flag, drains its own copies and MMAs (bounded), frees TMEM
// and returns.
#include <atomic>

#include "kv8.cuh"
#include "internal.h"
#include "warp_mma.cuh"

namespace pp {
namespace {

// Register split: launched with 128 a thread (512 * 128 = 65536); the control
// warps drop to 56, the converters to 72, the softmax warps rise to 192.
constexpr int kThreads8 = 512;
constexpr int kRegs8 = 128, kRegsCtl = 56, kRegsConv = 72, kRegsSoft = 192;
static_assert(128 * kRegsCtl + 128 * kRegsConv + 256 * kRegsSoft <= kThreads8 * kRegs8,
              "register split");
// Tiles of page scales kept (the loader runs at most 6 ahead of the softmax):
// for every 16 keys the key scale and the value scale's logarithm, -inf where
// there are no keys; [8]: whether any of the tile's keys are not there.
constexpr int kInfo = 8, kInfoLd = 9;
// Least factor of a score: a hidden one is -inf, and -inf * 0 would be NaN.
constexpr float kLeast = 1e-37f;

struct Doc8Params {
  pp_kv8_layer L;
  const uint16_t* q;
  int64_t q_ld;
  int g;        // query heads per key head
  int rows;     // (query row, query head) pairs of a key head
  int doc_len;
  SplitPlan plan;
  float sl2;
  float* doc_o;
  float* doc_ml;
  long long wait_limit;
  int inject_timeout;
};

template <int D>
struct Cfg8 {
  static constexpr int KH = D / 64;               // 128-byte column halves of an f16 row
  static constexpr int BOX = 128 * 64 * 2;        // [128 x 64] f16
  static constexpr int TILE = KH * BOX;           // f16 tile of queries, keys or values
  static constexpr int RAW = 128 * D;             // e4m3 tile
  static constexpr int NF = 4;                    // f16 key / value tiles (alternating)
  static constexpr int NR = D == 128 ? 1 : 2;     // e4m3 tiles of keys, and as many of values
  // Keys and values each by their own loader and two converting warps, or one
  // loader and four warps for both in turn.  Apart, a tile waits for nothing of
  // the other kind's, which pays where two tiles of a kind fit (d 64, 64 / 256
  // rows, 32768 keys: 92 -> 72 / 123 -> 117 us); with one (d 128: 107 -> 113 /
  // 130 -> 133) it costs more than it gives.
  static constexpr bool APART = NR > 1;
  static constexpr int CONV = APART ? 2 : 4;      // warps that convert a tile
  static constexpr int OFF_F = 2 * TILE;
  static constexpr int OFF_R = OFF_F + NF * TILE;
  static constexpr int OFF_INFO = OFF_R + 2 * NR * RAW;
  static constexpr int OFF_BAR = OFF_INFO + kInfo * kInfoLd * 8;
  // raw_full[2 NR], raw_empty[2 NR] (keys, values), f_full[NF], f_empty[NF], q_full[2], s_full[2],
  // p_full[2], o_done[2], drain
  static constexpr int NBAR = 4 * NR + 2 * NF + 9;
  static constexpr int USED = OFF_BAR + NBAR * 8 + 8;   // TMEM base and abort flag last
  // at least 120 KB so one CTA owns an SM's TMEM
  static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory above the per-CTA limit");
  static constexpr uint32_t T_S = 2 * D, TMEM_COLS = 512;
  static_assert(T_S + 2 * kBN <= TMEM_COLS, "TMEM budget");
};

// One arrival for a warp whose lanes have all done what the barrier stands for.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// 16-byte unit c of row r in a tile of 128-byte-swizzled rows of 64 f16.
__device__ __forceinline__ uint4* unit_at(uint8_t* tile, int r, int c) {
  return reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// A warp's 32 rows of queries (from pair `row0` on) to f16 in rows r0 .. r0 + 31
// of the swizzled tile, each a power of two smaller; returns that of the lane's
// row.  The rows come in whole, through their own place in the tile.  A NaN or
// infinity becomes NaN.
template <int D>
__device__ __forceinline__ float load_queries(const Doc8Params& p, uint8_t* tile, int r0, int row0,
                                              int h, int lane) {
  constexpr int U = D / 8, RP = 32 / U;   // units a row, rows a pass
  const uint16_t* head = p.q + (int64_t)h * p.g * D + (lane % U) * 8;
#pragma unroll 4
  for (int i = 0; i < 32; i += RP) {
    const int row = row0 + i + lane / U;
    const int at = row < p.rows ? row : 0;
    const int qr = p.g == 1 ? at : at / p.g;
    cp_async16(smem_u32(unit_at(tile, r0 + i + lane / U, lane % U)),
               head + (int64_t)qr * p.q_ld + (int64_t)(at - qr * p.g) * D, row < p.rows ? 16 : 0);
  }
  cp_async_wait_all();
  __syncwarp();
  const int r = r0 + lane;
  uint32_t am2 = 0;                       // largest magnitudes, as bits, of two columns
#pragma unroll 4
  for (int i = 0; i < U; ++i) {
    const uint4 x = *unit_at(tile, r, i);
    const uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("max.u16x2 %0, %0, %1;" : "+r"(am2) : "r"(a[j] & 0x7fff7fffu));
  }
  const uint32_t am = max(am2 & 0xffffu, am2 >> 16);
  // 2^e with the largest value / 2^e in [2^13, 2^14): bf16's 8 bits are exact in
  // f16 down to 2^-30 of it
  int e = (int)(am >> 7) - 127 - 13;
  e = e < -60 ? -60 : e;
  const float inv = am >= 0x7f80u ? __int_as_float(0x7fffffff)
                                  : __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 4
  for (int i = 0; i < U; ++i) {
    const uint4 x = *unit_at(tile, r, i);
    const uint32_t a[4] = {x.x, x.y, x.z, x.w};
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = bf2_to_f2(a[j]);
      b[j] = f2_to_h2(f.x * inv, f.y * inv);
    }
    *unit_at(tile, r, i) = make_uint4(b[0], b[1], b[2], b[3]);
  }
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <int D>
__global__ void __maxnreg__(kRegs8) kv8_doc_tc(const Doc8Params p) {
  using C = Cfg8<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  volatile int* abort_flag = reinterpret_cast<int*>(smem + C::OFF_BAR + C::NBAR * 8 + 4);
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + C::NBAR * 8);
  if (smem_u32(smem) & 1023) {     // (the swizzled tiles need it; never seen)
    set_status(p.L.status, PP_DEV_TIMEOUT);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* raw_full = bar;
  uint64_t* raw_empty = raw_full + 2 * C::NR;
  uint64_t* f_full = raw_empty + 2 * C::NR;
  uint64_t* f_empty = f_full + C::NF;
  uint64_t* q_full = f_empty + C::NF;
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 2;
  uint64_t* drain = o_done + 2;
  float2* info = reinterpret_cast<float2*>(smem + C::OFF_INFO);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const Runs8 runs = first_run8(p.plan, cta);
  int32_t* status = p.L.status;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * C::NR; ++i) {
      mbar_init(raw_full + i, 1);
      mbar_init(raw_empty + i, C::CONV);
    }
    for (int i = 0; i < C::NF; ++i) {
      mbar_init(f_full + i, C::CONV);
      mbar_init(f_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 4);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base;
  // the segment pass may fill SMs as this pass's CTAs end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0 || (C::APART && warp == 3)) {
    // ------------------------------------------------------------ loader ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    const int page = p.L.page, ppt = kBN / page;   // pages per tile
    const int groups = page >> 4;
    const int per = 32 / ppt;                      // tiles per batch of 32 pages, a lane each
    Runs8 t = runs;
    Seg8 s;
    const int kind = warp == 3;                    // where apart: 0 keys, 1 values
    int kt = 0, ht = 0;                            // tiles; copies this warp started
    bool ok = true;
    // Table entries are loaded two batches ahead, scales one, so that neither
    // dependent load stands between two tiles' copies.
    auto entry = [&](int b) {   // page b * 32 + lane of the document
      const int64_t i = (int64_t)b * 32 + lane;
      return i * page < p.doc_len ? p.L.doc_table[i] : -1;
    };
    auto scales = [&](int h, int pg, float& ks, float& vs) {
      ks = vs = 1.f;
      if (pg >= 0) {
        ks = p.L.k_scale[(int64_t)pg * p.L.H + h];
        vs = p.L.v_scale[(int64_t)pg * p.L.H + h];
      }
    };
    while (ok && next_seg8(p.plan, p.rows, t, s)) {
      int b = s.j0 / per;
      int pg0 = page_of(entry(b), p.L.n_pages), e1 = entry(b + 1);
      float ks0, vs0, ks1, vs1;
      scales(s.h, pg0, ks0, vs0);
      int pg1 = page_of(e1, p.L.n_pages);
      scales(s.h, pg1, ks1, vs1);
      e1 = entry(b + 2);
      for (int j = s.j0; ok && j < s.j0 + s.n; ++j, ++kt) {
        if (j / per != b) {
          b = j / per;
          pg0 = pg1; ks0 = ks1; vs0 = vs1;
          pg1 = page_of(e1, p.L.n_pages);
          scales(s.h, pg1, ks1, vs1);
          e1 = entry(b + 2);
        }
        const int from = (j % per) * ppt + (lane & 7);    // lanes 0 .. ppt-1 take the tile's pages
        const int pg = __shfl_sync(0xffffffffu, pg0, from & 31);
        const float ks = __shfl_sync(0xffffffffu, ks0, from & 31);
        const float vs = __shfl_sync(0xffffffffu, vs0, from & 31);
        const int64_t left = lane < ppt ? p.doc_len - ((int64_t)j * ppt + lane) * page : 0;
        if (left > 0 && pg < 0) set_status(status, PP_DEV_BAD_PAGE);
        // keys of this lane's page
        const int n = left > 0 && pg >= 0 ? (int)(left < page ? left : page) : 0;
        const uint32_t bytes = (uint32_t)n * D;
        uint32_t total = bytes;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total = __shfl_sync(0xffffffffu, total, 0);   // lanes 0..7 hold all pages of a tile
        const int64_t at = ((int64_t)(pg < 0 ? 0 : pg) * p.L.H + s.h) * page * D;
        const int sl = kt % C::NR, f = kt / C::NR;
        for (int x = 0; x < (C::APART ? 1 : 2); ++x) {
          const int kv = C::APART ? kind : x;
          uint64_t* full = raw_full + kv * C::NR + sl;
          if (f > 0 && !(ok = warp_wait(raw_empty + kv * C::NR + sl, (f - 1) & 1, abort_flag,
                                        p.wait_limit, status)))
            break;
          // (two loaders write the same scales: the softmax reads them behind the keys'
          // arrival, the values' converter behind the values')
          if ((C::APART || kv == 0) && lane < ppt) {
            for (int gq = 0; gq < groups; ++gq) {
              info[(kt % kInfo) * kInfoLd + lane * groups + gq] =
                  n > gq * 16 ? make_float2(ks, (float)((int)(__float_as_uint(vs) >> 23) - 127))
                              : make_float2(1.f, -INFINITY);
            }
          }
          if ((C::APART || kv == 0) && lane == 0)
            info[(kt % kInfo) * kInfoLd + 8].x = total < (uint32_t)(kBN * D) ? 1.f : 0.f;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full, total);
          __syncwarp();
          if (bytes && !(p.inject_timeout && kt + kv == 0))   // test hook: this copy never lands
            bulk_load(smem + C::OFF_R + (kv * C::NR + sl) * C::RAW + lane * page * D,
                      (kv ? p.L.v : p.L.k) + at, bytes, full);
          ++ht;
        }
      }
    }
    if (!ok && lane == 0) {
      // Drain: wait (bounded, abort flag ignored) for the copies still in flight.
      for (int back = 1; back <= (C::APART ? 1 : 2) * C::NR && ht - back >= 0; ++back) {
        const int kv = C::APART ? kind : (ht - back) & 1, k2 = C::APART ? ht - back : (ht - back) >> 1;
        if (p.inject_timeout && k2 + kv == 0) continue;
        volatile int never = 0;
        mbar_wait(raw_full + kv * C::NR + k2 % C::NR, (k2 / C::NR) & 1, &never, p.wait_limit,
                  nullptr);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    constexpr uint32_t IDESC_QK = idesc_f16_f32(128, kBN, 0);
    constexpr uint32_t IDESC_PV = idesc_f16_f32(128, D, 1);
    const uint32_t on = elect_one() ? 1u : 0u;   // one lane issues, always the same
    const uint64_t dQ = smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t dK = smem_desc_sw128(smem_u32(smem + C::OFF_F), 16, 1024);
    const uint64_t dV = smem_desc_sw128(smem_u32(smem + C::OFF_F), C::BOX, 1024);
    auto issue_qk = [&](int st, int slot) {
      const uint32_t d_t = tmem + C::T_S + (uint32_t)(st * kBN);
      const uint64_t a0 = dQ + (uint64_t)((st * C::TILE) >> 4);
      const uint64_t b0 = dK + (uint64_t)((slot * C::TILE) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4);
        mma_ss_if(on, d_t, a0 + off, b0 + off, IDESC_QK, kk > 0 ? 1u : 0u);
      }
    };
    auto issue_pv = [&](int st, int slot, bool acc) {
      const uint32_t d_t = tmem + (uint32_t)(st * D);
      const uint32_t a_t = tmem + C::T_S + (uint32_t)(st * kBN);
      const uint64_t b0 = dV + (uint64_t)((slot * C::TILE) >> 4);
#pragma unroll
      for (int kk = 0; kk < kBN / 16; ++kk)
        mma_ts_if(on, d_t, a_t + kk * 8, b0 + (uint64_t)((kk * 16 * 128) >> 4), IDESC_PV,
                  (acc || kk > 0) ? 1u : 0u);
    };
    auto commit = [&](uint64_t* b) { tc_commit_if(on, b); };
    auto wait_f = [&](int half) {
      return warp_wait(f_full + half % C::NF, (half / C::NF) & 1, abort_flag, p.wait_limit, status);
    };
    Runs8 t = runs;
    Seg8 s;
    int t0 = 0;
    uint32_t q_ph = 0, pf_ph = 0;   // bit st: the stream's parity
    bool ok = true;
    while (ok && next_seg8(p.plan, p.rows, t, s)) {
      const int step = s.two ? 1 : 2;
      for (int st = 0; ok && st < 2; ++st) {
        if (!has_tile8(s, st)) continue;
        if (!(ok = warp_wait(q_full + st, (q_ph >> st) & 1, abort_flag, p.wait_limit, status)))
          break;
        q_ph ^= 1u << st;
        const int tile = first_tile8(s, st);
        const int half = 2 * (t0 + tile);
        if (!(ok = wait_f(half))) break;
        tc_fence_after();
        issue_qk(st, half % C::NF);
        commit(s_full + st);
        if (!s.two || st == 1) commit(f_empty + half % C::NF);
      }
      const int steps = s.two ? 2 * s.n : s.n;
      for (int i = 0; ok && i < steps; ++i) {
        const int st = i & 1, tile = s.two ? i >> 1 : i;
        const int hv = 2 * (t0 + tile) + 1;
        if (!(ok = wait_f(hv))) break;
        if (!(ok = warp_wait(p_full + st, (pf_ph >> st) & 1, abort_flag, p.wait_limit, status))) break;
        pf_ph ^= 1u << st;
        tc_fence_after();
        issue_pv(st, hv % C::NF, tile >= step);
        if (!s.two || st == 1) commit(f_empty + hv % C::NF);
        if (tile + step < s.n) {
          // S is overwritten behind the product that reads P from it: the MMA
          // pipe runs in issue order
          const int hk = 2 * (t0 + tile + step);
          if (!(ok = wait_f(hk))) break;
          tc_fence_after();
          issue_qk(st, hk % C::NF);
          commit(s_full + st);
          if (!s.two || st == 1) commit(f_empty + hk % C::NF);
        } else {
          commit(o_done + st);
        }
      }
      t0 += s.n;
    }
    if (!ok) {
      commit(drain);
      if (lane == 0) {
        volatile int never = 0;
        mbar_wait(drain, 0, &never, p.wait_limit, nullptr);
      }
    }
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
  } else if (warp < 8) {
    // --------------------------------------------------------- converter ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    // A thread takes 16-byte unit u (16 dims) of every RS-th row from r0 on.  The
    // eight threads that access shared memory together take two rows, with u
    // dealt out so that their loads and both of their stores meet 32 different
    // banks.  RS is a multiple of 8: the swizzle is the same for all rows.
    constexpr int NT = C::CONV * 32, UR = D / 16, RS = NT / UR, IT = 128 / RS;
    const int kind = (warp - 4) >> 1, tid = threadIdx.x % NT;
    const int sub = tid & 7;
    const int u = D == 128 ? sub : sub & 3;
    const int r0 = D == 128 ? (tid >> 4) * 2 + ((sub >> 2) ^ ((tid >> 3) & 1)) : tid >> 2;
    const int src0 = r0 * D + u * 16;
    const int ua = (u & 3) * 2;
    const int dst0 = (u >> 2) * C::BOX + r0 * 128 + ((ua ^ (r0 & 7)) << 4);
    const int dst1 = (u >> 2) * C::BOX + r0 * 128 + (((ua + 1) ^ (r0 & 7)) << 4);
    Runs8 t = runs;
    Seg8 s;
    int kt = 0;
    bool ok = true;
    while (ok && next_seg8(p.plan, p.rows, t, s)) {
      for (int j = 0; ok && j < s.n; ++j, ++kt) {
        for (int x = 0; x < (C::APART ? 1 : 2); ++x) {
          const int kv = C::APART ? kind : x;
          const int sr = kv * C::NR + kt % C::NR, ft = 2 * kt + kv, sf = ft % C::NF;
          if (!(ok = warp_wait(raw_full + sr, (kt / C::NR) & 1, abort_flag, p.wait_limit, status)))
            break;
          if (ft >= C::NF && !(ok = warp_wait(f_empty + sf, (ft / C::NF - 1) & 1, abort_flag,
                                              p.wait_limit, status)))
            break;
          const uint8_t* src = smem + C::OFF_R + sr * C::RAW + src0;
          uint8_t* dst = smem + C::OFF_F + sf * C::TILE;
          uint4 w[IT];
#pragma unroll
          for (int i = 0; i < IT; ++i) w[i] = *reinterpret_cast<const uint4*>(src + i * RS * D);
          const float2* inf = info + (kt % kInfo) * kInfoLd;
          if (inf[8].x != 0.f) {      // some keys are not there: zeros for them (rare)
            const int there = p.doc_len - (s.j0 + j) * kBN;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
              const int r = r0 + i * RS;
              if (r >= there || inf[r >> 4].y == -INFINITY) w[i] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            *reinterpret_cast<uint4*>(dst + dst0 + i * RS * 128) =
                make_uint4(e4m3x2_to_h2(w[i].x), e4m3x2_hi_to_h2(w[i].x), e4m3x2_to_h2(w[i].y),
                           e4m3x2_hi_to_h2(w[i].y));
            *reinterpret_cast<uint4*>(dst + dst1 + i * RS * 128) =
                make_uint4(e4m3x2_to_h2(w[i].z), e4m3x2_hi_to_h2(w[i].z), e4m3x2_to_h2(w[i].w),
                           e4m3x2_hi_to_h2(w[i].w));
          }
          // behind the stores, which need the loaded values: with the arrival right
          // behind the loads the next copy was seen to overtake them
          fence_proxy_async();
          warp_arrive(raw_empty + sr, lane);
          warp_arrive(f_full + sf, lane);
        }
      }
    }
  } else {
    // ----------------------------------------------------------- softmax ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int st = (warp - 8) >> 2;
    const int wq = warp & 3;                 // TMEM lane quarter of this warp
    const int rt = wq * 32 + lane;           // row of the M tile
    const uint32_t t_lane = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t t_S = t_lane + C::T_S + (uint32_t)(st * kBN);
    const uint32_t t_O = t_lane + (uint32_t)(st * D);
    uint8_t* tq = smem + st * C::TILE;
    Runs8 t = runs;
    Seg8 s;
    uint32_t s_ph = 0, od_ph = 0;
    int t0 = 0;
    bool ok = true;
    while (ok && next_seg8(p.plan, p.rows, t, s)) {
      const int step = s.two ? 1 : 2, first = first_tile8(s, st);
      const bool tiles = has_tile8(s, st);
      const int row = s.gi * kGroupRows + (s.two ? st * 128 : 0) + rt;
      // (the previous run's last S has been seen: no MMA reads this tile of Q any more)
      float qs = 0.f;
      if (tiles) {
        qs = load_queries<D>(p, tq, wq * 32, row - lane, s.h, lane) * p.sl2;
        fence_proxy_async();
        warp_arrive(q_full + st, lane);
      }
      float m = 0.f, l = 0.f;
      bool none = true;                        // no key so far
      for (int tile = first; tile < s.n; tile += step) {
        if (!(ok = warp_wait(s_full + st, s_ph, abort_flag, p.wait_limit, status))) break;
        s_ph ^= 1;
        const float2* inf = info + ((t0 + tile) % kInfo) * kInfoLd;
        tc_fence_after();
        const int kvalid = p.doc_len - (s.j0 + tile) * kBN;
        if (kvalid < kBN) {              // the document's last tile: hide what is behind it
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(t_S + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= kvalid) x[e] = __float_as_uint(-INFINITY);
            tmem_st32(t_S + c * 32, x);
          }
          tmem_st_wait();
        }
        // the row's maximum of w
        auto maximum = [&]() {
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(t_S + c * 32, x);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float2 in = inf[c * 2 + q];
              float y = __uint_as_float(x[q * 16]);
#pragma unroll
              for (int e = 1; e < 16; ++e) y = fmaxf(y, __uint_as_float(x[q * 16 + e]));
              mx = fmaxf(mx, fmaf(y, fmaxf(in.x * qs, kLeast), in.y));
            }
          }
          return mx;
        };
        uint32_t pk[64];
        float lt, sum;
        // P of the tile, its sum, and the sum over the value scales
        auto exponentials = [&]() {
          lt = sum = 0.f;
          uint32_t r[2][32];
          float2 in[2][2];                 // scales of 2 x 16 keys, and of the next
          in[0][0] = inf[0];
          in[0][1] = inf[1];
          tmem_ld32(t_S, r[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_wait();
            if (c < 3) {
              tmem_ld32(t_S + (c + 1) * 32, r[(c + 1) & 1]);
              in[(c + 1) & 1][0] = inf[c * 2 + 2];
              in[(c + 1) & 1][1] = inf[c * 2 + 3];
            }
            uint32_t (&x)[32] = r[c & 1];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float a = fmaxf(in[c & 1][q].x * qs, kLeast), g = in[c & 1][q].y, b = g - m;
              const float rv = g == -INFINITY ? 0.f : ex2_mufu(-g);   // 1 / value scale
              const float2 av = make_float2(a, a), bv = make_float2(b, b);
              float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float2 w = ffma2(make_float2(__uint_as_float(x[q * 16 + e]),
                                                   __uint_as_float(x[q * 16 + e + 1])), av, bv);
                // one in four on the FMA pipe (1/8, 1/4, 5/16, 3/8 of them: 1490 / 1511 /
                // 1536 / 1599 us of a question prefill of 8192 rows, 12000 keys; decode of
                // 256 rows, 16384 keys 133 / 130 / 130 / 131)
                const float2 pv = (e >> 1) % 4 == 1
                                      ? ex2_poly2_wide(w)
                                      : make_float2(ex2_mufu(w.x), ex2_mufu(w.y));
                rs[(e >> 1) & 1] = fadd2(rs[(e >> 1) & 1], pv);
                pk[c * 16 + q * 8 + (e >> 1)] = f2_to_h2(pv.x, pv.y);
              }
              const float2 r2 = fadd2(rs[0], rs[1]);
              const float r1 = r2.x + r2.y;
              sum += r1;
              lt = fmaf(r1, rv, lt);
            }
          }
        };
        // Rows without a reference yet, or whose sum says that it is too low, take
        // their maximum first (the warp does, for all its rows; the others keep
        // theirs).  The product of this stream's tile before is complete: it was
        // issued ahead of this S.
        sum = 0.f;
        bool raise = __any_sync(0xffffffffu, none);
        for (int tries = 0;; ++tries) {
          if (raise) {
            const float mx = maximum();
            const bool move = none ? mx != -INFINITY : sum > 4096.f;
            const float f = !move ? 1.f : none ? 0.f : ex2_mufu(m - mx);
            if (move) {
              m = mx;
              l *= f;
              none = false;
            }
            if (tile > first) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(t_O + c * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(t_O + c * 32, o);
              }
            }
          }
          exponentials();
          if (tries == 2 || !__any_sync(0xffffffffu, sum > 4096.f)) break;
          raise = true;
        }
        // A NaN score: the sum is NaN, or, from the polynomial, still huge.
        if (sum > 1e18f || sum != sum) lt = __int_as_float(0x7fffffff);
        none = none && lt == lt;
        l += lt;
        tmem_st32(t_S, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st32(t_S + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(p_full + st, lane);
      }
      if (!ok) break;
      // partial of this run: the unit's first CTA has chunk 0
      const int chunk =
          s.j0 == 0 ? 0 : cta - plan_cta_of(p.plan, (int64_t)s.u * p.plan.T + kKv8Lead);
      const int64_t prow = ((int64_t)s.u * p.plan.max_chunks + chunk) * kGroupRows + st * 128 + rt;
      if (tiles) {
        if (!(ok = warp_wait(o_done + st, od_ph, abort_flag, p.wait_limit, status))) break;
        od_ph ^= 1;
        tc_fence_after();
        // through the rows' place in the query tile, so that rows go out in whole
        // sectors
        float* dst = p.doc_o + (prow - lane) * D;
        const int n_rows = p.rows - (row - lane);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_O + c * 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *unit_at(tq, rt, e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          __syncwarp();
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = *unit_at(tq, wq * 32 + i * 4 + (lane >> 3), lane & 7);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i * 4 + (lane >> 3) < n_rows)
              *reinterpret_cast<uint4*>(dst + (i * 4 + (lane >> 3)) * D + c * 32 + (lane & 7) * 4) = w[i];
          __syncwarp();
        }
        tc_fence_before();
      }
      // a NaN row keeps a finite maximum so that the merge does not skip it
      if (row < p.rows)
        reinterpret_cast<float2*>(p.doc_ml)[prow] = make_float2(none ? -INFINITY : m, l);
      t0 += s.n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D>
cudaError_t launch(const Doc8Params& p, cudaStream_t st) {
  using C = Cfg8<D>;
  // Once per device: allow the dynamic shared memory, and check that the
  // kernel was built with the register count the split assumes (with fewer the
  // softmax warps' increase would wait forever).
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kv8_doc_tc<D>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegs8) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kv8_doc_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  kv8_doc_tc<D><<<p.plan.C, kThreads8, C::SMEM, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_doc(const pp_kv8_layer& L, const pp_kv8_attn_args& a, const SplitPlan& plan,
                           const Partials& part, long long wait_limit, int inject_timeout,
                           cudaStream_t st) {
  Doc8Params p{};
  p.L = L;
  p.q = a.q; p.q_ld = a.q_ld;
  p.g = a.Hq / L.H;
  p.rows = a.rows * p.g;
  p.doc_len = a.doc_len;
  p.plan = plan;
  p.sl2 = a.scale * kLog2e;
  p.doc_o = part.doc_o; p.doc_ml = part.doc_ml;
  p.wait_limit = wait_limit;
  p.inject_timeout = inject_timeout;
  return L.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace pp
