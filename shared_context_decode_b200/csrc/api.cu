// C-ABI entry points of libppattn (declared in include/ppattn.h).
//
// Host code here validates arguments, derives the document split plan,
// carves the caller's workspace and launches the kernels in stream order:
//   decode / prefill:  [document pass] -> suffix pass with the merge fused
// Nothing here allocates device memory or synchronises (except
// pp_get_device_status), so the calls can be captured in a CUDA graph.
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "kv8.cuh"

namespace {

using pp::Partials;
using pp::SplitPlan;

constexpr size_t kAlign = 256;

size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && cache[dev].load() > 0) return cache[dev].load();
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) cache[dev].store(n);
  return n;
}

}  // namespace

namespace pp {
pp_status check_layer(const pp_kv_layer* L) {
  if (!L) return PP_ERR_INVALID_ARG;
  if (L->d != 64 && L->d != 128) return PP_ERR_UNSUPPORTED;
  if (L->P_max < 1 || L->P_max > 32767) return PP_ERR_UNSUPPORTED;
  if (L->H < 1 || L->doc_cap < 0 || L->S_cap < 1) return PP_ERR_INVALID_ARG;
  if (L->doc_cap > 0 && (!L->k_doc || !L->v_doc || !aligned(L->k_doc, 16) || !aligned(L->v_doc, 16)))
    return PP_ERR_INVALID_ARG;
  if (!L->k_suf || !L->v_suf || !aligned(L->k_suf, 16) || !aligned(L->v_suf, 16))
    return PP_ERR_INVALID_ARG;
  if (!L->sid || !L->pos || !L->len || !L->status || !aligned(L->sid, 2) || !aligned(L->pos, 4) ||
      !aligned(L->len, 4) || !aligned(L->status, 4))
    return PP_ERR_INVALID_ARG;
  return PP_OK;
}
}  // namespace pp

namespace {
using pp::check_layer;

pp_status from_cuda(cudaError_t e) { return e == cudaSuccess ? PP_OK : PP_ERR_CUDA; }

// A named NVTX range around an entry point, so a profiler's timeline shows
// each C-ABI call (header-only NVTX: without an attached tool a push/pop is
// a check of a null function pointer).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// The document split: see pp::SplitPlan.  `ctas` = slots to spread it over;
// `causal`: a document prefill (rows = document tokens, triangular units).
SplitPlan make_plan(int rows, int H, int doc_len, int ctas, bool causal = false) {
  SplitPlan p{};
  p.T = (doc_len + pp::kBN - 1) / pp::kBN;
  p.G = (rows + pp::kGroupRows - 1) / pp::kGroupRows;
  p.units = p.G * H;
  p.causal = causal ? 1 : 0;
  p.W = p.G > 0 && p.T > 0 ? (int64_t)H * pp::plan_head_tiles(p) : 0;
  if (p.W == 0 || ctas < 1) {
    p.C = 0;
    p.max_chunks = 0;
    return p;
  }
  p.C = (int32_t)std::min<int64_t>(ctas, p.W);
  int mc = 1;
  for (int u = 0; u < p.units; ++u) {
    const int64_t ub = pp::plan_unit_begin(p, u);
    const int n = pp::plan_cta_of(p, ub + pp::plan_unit_tiles(p, u % p.G) - 1) -
                  pp::plan_cta_of(p, ub) + 1;
    mc = std::max(mc, n);
  }
  p.max_chunks = mc;
  return p;
}

// The ablation reads the whole document per row: one chunk per unit.
SplitPlan ablation_plan(int rows, int H, int doc_len) {
  SplitPlan p{};
  p.G = (rows + pp::kGroupRows - 1) / pp::kGroupRows;
  p.units = p.G * H;
  p.T = doc_len > 0 ? 1 : 0;
  p.W = (int64_t)p.units * p.T;
  p.C = (int32_t)p.W;
  p.max_chunks = p.W > 0 ? 1 : 0;
  return p;
}

SplitPlan plan_for(int rows, int H, int doc_len, const pp_options* opt, bool causal = false) {
  if (opt && opt->ablation_doc_per_stream && !causal) return ablation_plan(rows, H, doc_len);
  // one slot (a CTA per M tile of a row group) per SM pair by default
  const int ctas = (opt && opt->splits > 0) ? opt->splits
                                           : std::max(1, sm_count() / pp::doc_pair_ctas(rows));
  return make_plan(rows, H, doc_len, ctas, causal);
}

struct WsLayout {
  size_t doc_o, doc_ml, row_len, split_cnt, split_o, split_ml, runs, n_runs, total;
};

// The document pass leaves its partial results in the workspace.  Besides,
// for decode and question prefill (not the causal document prefill): each
// row's stream length when the pass carries a decode step's append, and the
// decode suffix pass's counters and partials for items cut between warps;
// question prefill (questions = true): the question runs (at most one per
// row), their count and the question kernel's task counter.
WsLayout ws_layout(const SplitPlan& p, int d, bool questions) {
  WsLayout w;
  const size_t slots = (size_t)p.units * p.max_chunks * pp::kGroupRows;
  const bool extra = slots && !p.causal;
  const size_t warps = extra ? (size_t)std::max(sm_count(), 0) * pp::kSuffixWarps : 0;
  w.doc_o = 0;
  w.doc_ml = w.doc_o + up(slots * d * sizeof(float));
  w.row_len = w.doc_ml + up(slots * 2 * sizeof(float));
  w.split_cnt = w.row_len + (extra ? up((size_t)p.G * pp::kGroupRows * sizeof(int32_t)) : 0);
  w.split_o = w.split_cnt + up(warps * sizeof(int32_t));
  w.split_ml = w.split_o + up(2 * warps * d * sizeof(float));
  w.runs = w.split_ml + up(2 * warps * 2 * sizeof(float));
  w.n_runs = w.runs + (questions ? up((size_t)p.G * pp::kGroupRows * sizeof(int4)) : 0);
  w.total = w.n_runs + (questions ? up(2 * sizeof(int32_t)) : 0);
  return w;
}

// Largest decode step whose append runs inside the document pass: every
// appended row counts its stream's rows over the whole call.
constexpr int kFusedAppendMaxRows = 4096;

Partials carve(void* ws, const WsLayout& w) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  Partials p;
  p.doc_o = reinterpret_cast<float*>(b + w.doc_o);
  p.doc_ml = reinterpret_cast<float*>(b + w.doc_ml);
  return p;
}

long long wait_limit(const pp_options* opt) {
  const int lg = (opt && opt->wait_limit_log2 > 0) ? std::min(opt->wait_limit_log2, 40) : 31;
  return 1LL << lg;
}

// Inside a stream capture the events become event-record nodes of the graph
// (recorded at every replay), so per-kernel timing also works for graphs.
cudaError_t record_mark(cudaEvent_t ev, cudaStreamCaptureStatus cap, cudaStream_t st) {
  return cap == cudaStreamCaptureStatusActive
             ? cudaEventRecordWithFlags(ev, st, cudaEventRecordExternal)
             : cudaEventRecord(ev, st);
}

// Shared body of decode and prefill attention.
// causal: a document prefill; rows = doc_len document tokens, no stream ids.
// app_k, app_v: a decode step's new keys and values (one row per query row,
// the rows' own stream ids and positions), appended before the attention:
// inside the document pass launch when there is one, else by the append
// kernels; nullptr: nothing to append.
// read_once: a decode step (one row per stream), so each segment is read once
// and the per-row suffix kernel runs; otherwise rows come in question-sized
// runs of one stream and the question-block kernel runs.
pp_status attend(const pp_kv_layer* L, int32_t doc_len, const uint16_t* q, const int16_t* q_sid,
                 const int32_t* q_pos, int32_t rows, float scale, uint16_t* o, float* lse, void* ws,
                 size_t ws_bytes, const pp_options* opt, void* stream, bool causal = false,
                 bool read_once = false, const uint16_t* app_k = nullptr,
                 const uint16_t* app_v = nullptr) {
  pp_status s = check_layer(L);
  if (s != PP_OK) return s;
  if (rows < 0 || doc_len < 0) return PP_ERR_INVALID_ARG;
  if (doc_len > L->doc_cap) return PP_ERR_CAPACITY;
  if (rows == 0) return PP_OK;
  if (!q || !o || !aligned(q, 16) || !aligned(o, 16) || (lse && !aligned(lse, 4)))
    return PP_ERR_INVALID_ARG;
  if (!causal && (!q_sid || !q_pos || !aligned(q_sid, 2) || !aligned(q_pos, 4)))
    return PP_ERR_INVALID_ARG;
  if (!(scale == scale)) return PP_ERR_INVALID_ARG;
  if (opt && (opt->suffix_slices < 0 || opt->suffix_slices > 2)) return PP_ERR_INVALID_ARG;
  if (causal && opt && (opt->ablation_doc_per_stream || opt->sibling_scan))
    return PP_ERR_UNSUPPORTED;
  const SplitPlan plan = plan_for(rows, L->H, doc_len, opt, causal);
  const bool has_doc = doc_len > 0;
  if (has_doc && plan.C < 1) return PP_ERR_CUDA;  // no device to size the split for
  const WsLayout w = ws_layout(plan, L->d, !causal && !read_once);
  if (w.total > 0 && (!ws || !aligned(ws, kAlign))) return PP_ERR_INVALID_ARG;
  if (ws_bytes < w.total) return PP_ERR_CAPACITY;
  const int sms = sm_count();
  if (sms < 1) return PP_ERR_CUDA;
  const Partials part = carve(ws, w);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaEvent_t* ev = (opt && opt->events) ? reinterpret_cast<cudaEvent_t*>(opt->events) : nullptr;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (ev && cudaStreamIsCapturing(st, &cap) != cudaSuccess) return PP_ERR_CUDA;
  auto mark = [&](int i) { return ev ? record_mark(ev[i], cap, st) : cudaSuccess; };
  const bool other_doc = opt && (opt->ablation_doc_per_stream || opt->sibling_scan);
  // decode behind the tensor-core document pass: the suffix slices are
  // balanced by work, with counters that pass zeroes
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  pp::SuffixSplit split{};
  // automatic: when equal item counts would leave most warps idle (items
  // for fewer than half of them) or a few long segments could hold most of
  // the work.  (With about one item per warp equal counts measured faster:
  // 22.5 against 26.7 us at 64 streams x 32 heads over 8192 document keys.)
  const int slices = opt ? opt->suffix_slices : 0;
  const bool want = slices == 2 ||
                    (slices == 0 && (2LL * rows * L->H < (int64_t)sms * pp::kSuffixWarps ||
                                     L->S_cap > 32 * 16));
  const bool balance = want && read_once && has_doc && !other_doc && rows <= pp::kBalanceRows &&
                       (int64_t)rows * L->H < (1LL << 31);
  if (balance) {
    split.cnt = reinterpret_cast<int32_t*>(wsb + w.split_cnt);
    split.o = reinterpret_cast<float*>(wsb + w.split_o);
    split.ml = reinterpret_cast<float*>(wsb + w.split_ml);
  }
  pp::AppendJob app{};
  if (app_k) {
    if (has_doc && !other_doc && rows <= kFusedAppendMaxRows) {
      app = {app_k, app_v, q_sid, q_pos, rows, reinterpret_cast<int32_t*>(wsb + w.row_len)};
    } else if ((s = from_cuda(pp::launch_kv_append(*L, app_k, app_v, q_sid, q_pos, rows, st,
                                                   true))) != PP_OK) {
      return s;
    }
  }
  if (mark(0) != cudaSuccess) return PP_ERR_CUDA;
  if (has_doc) {
    cudaError_t e;
    if (opt && opt->ablation_doc_per_stream)
      e = pp::launch_doc_per_stream(*L, doc_len, q, rows, scale, plan.max_chunks, part, st);
    else
      e = pp::launch_doc_pass_tc(*L, doc_len, q, rows, scale, plan, part, wait_limit(opt),
                                 opt ? opt->debug_inject_timeout : 0, app, split.cnt,
                                 balance ? sms * pp::kSuffixWarps : 0, st);
    if (e != cudaSuccess) return PP_ERR_CUDA;
  }
  if (mark(1) != cudaSuccess) return PP_ERR_CUDA;
  if (opt && opt->sibling_scan) {
    if ((s = from_cuda(pp::launch_sibling_scan(*L, q, q_sid, q_pos, rows, scale, plan, has_doc,
                                               part, o, lse, st))) != PP_OK)
      return s;
  } else if (read_once) {
    if ((s = from_cuda(pp::launch_suffix_merge(*L, q, q_sid, q_pos, rows, scale, plan, has_doc,
                                               part, o, lse, wait_limit(opt), sms,
                                               app.n ? app.row_len : nullptr,
                                               balance ? &split : nullptr, st))) != PP_OK)
      return s;
  } else if (!causal) {
    int4* runs = reinterpret_cast<int4*>(wsb + w.runs);
    int32_t* n_runs = reinterpret_cast<int32_t*>(wsb + w.n_runs);
    if ((s = from_cuda(pp::launch_question_runs(*L, q_sid, rows, runs, n_runs, st))) != PP_OK)
      return s;
    if ((s = from_cuda(pp::launch_question_attn(*L, q, q_sid, q_pos, rows, scale, plan, has_doc,
                                                part, o, lse, runs, n_runs, sms, st))) != PP_OK)
      return s;
  } else if ((s = from_cuda(pp::launch_doc_merge(rows, L->H, L->d, plan, part, o, lse, st))) !=
             PP_OK) {
    return s;  // a document prefill: its rows see the document only
  }
  return from_cuda(mark(2));
}

// questions: a question prefill (pp_prefill_attn), whose question runs
// need room whether or not there is a document.
size_t workspace(int32_t rows, int32_t H, int32_t d, int32_t doc_len, const pp_options* opt,
                 bool causal = false, bool questions = false) {
  if (rows < 0 || H < 1 || (d != 64 && d != 128) || doc_len < 0) return 0;
  const SplitPlan plan = plan_for(rows, H, doc_len, opt, causal);
  if (doc_len > 0 && plan.C < 1) return 0;
  return ws_layout(plan, d, questions).total;
}

// ------------------------------------------------ 8-bit paged cache ----
pp_status check_kv8_layer(const pp_kv8_layer* L) {
  if (!L) return PP_ERR_INVALID_ARG;
  if (L->d != 64 && L->d != 128) return PP_ERR_UNSUPPORTED;
  if (L->page != 16 && L->page != 32 && L->page != 64 && L->page != 128) return PP_ERR_UNSUPPORTED;
  if (L->P_max < 1 || L->P_max > 32767) return PP_ERR_UNSUPPORTED;
  if (L->H < 1 || L->n_pages < 1 || L->seg_pages < 1 || L->doc_pages < 0 || L->pos0 < 0)
    return PP_ERR_INVALID_ARG;
  // positions and (page, head) cells are 32-bit numbers
  const int64_t most = INT32_MAX - 256;
  if ((int64_t)L->pos0 + (int64_t)L->seg_pages * L->page > most ||
      (int64_t)L->doc_pages * L->page > most || (int64_t)L->n_pages * L->H > most)
    return PP_ERR_UNSUPPORTED;
  if (!L->k || !L->v || !aligned(L->k, 16) || !aligned(L->v, 16)) return PP_ERR_INVALID_ARG;
  if (!L->k_scale || !L->v_scale || !aligned(L->k_scale, 4) || !aligned(L->v_scale, 4))
    return PP_ERR_INVALID_ARG;
  if (!L->seg_table || !aligned(L->seg_table, 4) ||
      (L->doc_pages > 0 && (!L->doc_table || !aligned(L->doc_table, 4))))
    return PP_ERR_INVALID_ARG;
  if (!L->status || !aligned(L->status, 4)) return PP_ERR_INVALID_ARG;
  return PP_OK;
}

// A strided row operand: heads packed, rows ld elements apart.
bool row_operand(const void* ptr, int64_t ld, int64_t heads, int32_t d) {
  return ptr && aligned(ptr, 16) && ld % 8 == 0 && ld >= heads * d;
}

// Split of the document over the tensor-core pass's CTAs; C = 0: the document
// is read by the segment kernel's warps instead (no pass, no workspace), which
// is faster while both its work and a warp's share of one document are small.
// Measured on either side (us, pass / warps): 16 rows, 8 heads, 2048 keys 21.3 /
// 18.8, 64 rows, 8 heads, 1024 keys 18.0 / 26.0; one row of one head, 16384
// keys 57 / 92, 4 rows of 4 heads, 4096 keys 25.0 / 28.7, 1024 keys 14.1 / 12.6.
SplitPlan kv8_plan(int32_t rows, int32_t Hq, int32_t H, int32_t doc_len, const pp_options* opt,
                   bool decode, int sms) {
  const int64_t items = pp::kv8_items(rows, Hq / H, H, decode).items;
  const bool asked = opt && (opt->splits > 0 || opt->debug_inject_timeout);
  if (rows == 0 || doc_len == 0 || (!asked && doc_len <= 3000 && items * doc_len <= 400000))
    return SplitPlan{};
  int ctas = asked && opt->splits > 0 ? opt->splits : sms;
  SplitPlan p{};
  p.T = (doc_len + pp::kBN - 1) / pp::kBN + pp::kKv8Lead;
  p.G = (rows * (Hq / H) + pp::kGroupRows - 1) / pp::kGroupRows;
  p.units = p.G * H;
  p.W = (int64_t)p.units * p.T;
  // few units: not so many parts that joining them takes longer than a part
  // (16384 keys, one row: 56 us in 148 parts, 31 in 16, 37 in 8; 4096 keys, 4
  // rows: 25, 24 and 21)
  if (!asked) {
    int parts = 1;
    while (parts * parts < 2 * p.T) ++parts;
    ctas = (int)std::min<int64_t>(ctas, (int64_t)parts * p.units);
  }
  // (46340^2 < 2^31: the kernel's products of two CTA counts hold in 32 bits)
  p.C = (int32_t)std::min<int64_t>(std::min(std::max(ctas, 0), 46340), p.W);
  if (p.C < 1) return SplitPlan{};
  // a unit's steps lie in at most this many CTAs' ranges of floor(W / C) or one more
  const int64_t least = p.W / p.C;
  p.max_chunks = (int32_t)((p.T - 2) / least + 2);
  return p;
}

WsLayout kv8_ws_layout(const SplitPlan& p, int d) {
  WsLayout w{};
  const size_t slots = p.C > 0 ? (size_t)p.units * p.max_chunks * pp::kGroupRows : 0;
  w.doc_ml = up(slots * d * sizeof(float));
  w.total = w.doc_ml + up(slots * 2 * sizeof(float));
  return w;
}

pp_status kv8_append(const pp_kv8_layer* L, const pp_kv8_append_args* a, void* stream) {
  pp_status s = check_kv8_layer(L);
  if (s != PP_OK) return s;
  if (!a || a->n < 0) return PP_ERR_INVALID_ARG;
  const pp_rope* rope = a->rope;
  if (rope) {
    if (rope->dim < 0 || rope->max_pos < 1 || !rope->cos_sin || !aligned(rope->cos_sin, 16))
      return PP_ERR_INVALID_ARG;
    if (rope->dim == 0 || rope->dim % 16 != 0 || rope->dim > L->d) return PP_ERR_UNSUPPORTED;
    if (rope->interleaved != 0 && rope->interleaved != 1) return PP_ERR_INVALID_ARG;
  }
  if (a->n == 0) return PP_OK;
  if (!row_operand(a->k, a->k_ld, L->H, L->d) || !row_operand(a->v, a->v_ld, L->H, L->d) ||
      !a->sid || !a->pos || !aligned(a->sid, 2) || !aligned(a->pos, 4))
    return PP_ERR_INVALID_ARG;
  if (!a->q != !a->q_out) return PP_ERR_INVALID_ARG;
  if (a->q && (a->Hq < 1 || a->Hq > (1 << 17) || !row_operand(a->q, a->q_ld, a->Hq, L->d) ||
               !row_operand(a->q_out, a->q_out_ld, a->Hq, L->d)))
    return PP_ERR_INVALID_ARG;
  if (L->H > (1 << 14)) return PP_ERR_UNSUPPORTED;    // blocks along y
  const int sms = sm_count();
  if (sms < 1) return PP_ERR_CUDA;
  return from_cuda(pp::launch_kv8_append(*L, *a, sms, static_cast<cudaStream_t>(stream)));
}

pp_status kv8_attend(const pp_kv8_layer* L, const pp_kv8_attn_args* a, void* stream, bool decode) {
  pp_status s = check_kv8_layer(L);
  if (s != PP_OK) return s;
  if (!a) return PP_ERR_INVALID_ARG;
  const int32_t rows = a->rows, doc_len = a->doc_len, Hq = a->Hq;
  const float scale = a->scale;
  const pp_options* opt = a->opt;
  if (rows < 0 || doc_len < 0 || Hq < 1 || Hq % L->H != 0) return PP_ERR_INVALID_ARG;
  if (decode && rows > L->P_max) return PP_ERR_UNSUPPORTED;
  if ((int64_t)doc_len > (int64_t)L->doc_pages * L->page) return PP_ERR_CAPACITY;
  if (opt && (opt->ablation_doc_per_stream || opt->sibling_scan || opt->suffix_slices))
    return PP_ERR_UNSUPPORTED;
  if (!(scale > 0.f) || scale > 3.4e38f) return PP_ERR_INVALID_ARG;
  if (rows == 0) return PP_OK;
  if (!row_operand(a->q, a->q_ld, Hq, L->d) || !a->o || !aligned(a->o, 16) ||
      (a->lse && !aligned(a->lse, 4)) || !a->q_sid || !a->q_pos || !aligned(a->q_sid, 2) ||
      !aligned(a->q_pos, 4))
    return PP_ERR_INVALID_ARG;
  if ((int64_t)rows * Hq > INT32_MAX - 256) return PP_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms < 1) return PP_ERR_CUDA;
  const SplitPlan plan = kv8_plan(rows, Hq, L->H, doc_len, opt, decode, sms);
  const bool doc_pass = plan.C > 0;
  // both kernels count in 32 bits
  if (plan.W > INT32_MAX ||
      pp::kv8_items(rows, Hq / L->H, L->H, decode).items > INT32_MAX / 16)
    return PP_ERR_UNSUPPORTED;
  const WsLayout w = kv8_ws_layout(plan, L->d);
  if (w.total > 0 && (!a->ws || !aligned(a->ws, kAlign))) return PP_ERR_INVALID_ARG;
  if (a->ws_bytes < w.total) return PP_ERR_CAPACITY;
  const Partials part = carve(a->ws, w);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaEvent_t* ev = (opt && opt->events) ? reinterpret_cast<cudaEvent_t*>(opt->events) : nullptr;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (ev && cudaStreamIsCapturing(st, &cap) != cudaSuccess) return PP_ERR_CUDA;
  auto mark = [&](int i) { return ev ? record_mark(ev[i], cap, st) : cudaSuccess; };
  if (mark(0) != cudaSuccess) return PP_ERR_CUDA;
  if (doc_pass && (s = from_cuda(pp::launch_kv8_doc(*L, *a, plan, part, wait_limit(opt),
                                                    opt ? opt->debug_inject_timeout : 0, st))) !=
                      PP_OK)
    return s;
  if (mark(1) != cudaSuccess) return PP_ERR_CUDA;
  if ((s = from_cuda(pp::launch_kv8_attn(*L, *a, decode, plan, doc_pass, part, sms, st))) != PP_OK)
    return s;
  return from_cuda(mark(2));
}

size_t kv8_workspace(int32_t rows, int32_t Hq, int32_t H, int32_t d, int32_t doc_len,
                     const pp_options* opt, bool decode) {
  if (rows < 0 || H < 1 || Hq < 1 || Hq % H != 0 || (d != 64 && d != 128) || doc_len < 0) return 0;
  if ((int64_t)rows * Hq > INT32_MAX - 256) return 0;
  return kv8_ws_layout(kv8_plan(rows, Hq, H, doc_len, opt, decode, sm_count()), d).total;
}

// The document pass's runs of every CTA, as the kernel's roles walk them.
pp_status write_kv8_runs(const SplitPlan& p, int rows, const pp::Kv8Items& items, int64_t* h_out,
                         int32_t h_out_len) {
  if (h_out_len < 8) return PP_ERR_CAPACITY;
  const int64_t head[8] = {p.T, p.units, p.W, p.C, p.max_chunks, items.most, items.items, 0};
  for (int i = 0; i < 8; ++i) h_out[i] = head[i];
  int64_t runs = 0;
  for (int cta = 0; cta < p.C; ++cta) {
    pp::Runs8 r = pp::first_run8(p, cta);
    pp::Seg8 s;
    for (; pp::next_seg8(p, rows, r, s); ++runs) {
      if (8 + 6 * (runs + 1) > h_out_len) return PP_ERR_CAPACITY;
      const int64_t run[6] = {cta, s.u, s.j0, s.n, s.two,
                              (int)pp::has_tile8(s, 0) + 2 * (int)pp::has_tile8(s, 1)};
      for (int i = 0; i < 6; ++i) h_out[8 + 6 * runs + i] = run[i];
    }
  }
  h_out[7] = runs;
  return PP_OK;
}

// Host copy of a plan for the split-plan test aids.
pp_status write_plan(const SplitPlan& p, int64_t* h_out, int32_t h_out_len) {
  if (h_out_len < 5 + 2 * (int64_t)p.units) return PP_ERR_CAPACITY;
  h_out[0] = p.T;
  h_out[1] = p.units;
  h_out[2] = p.W;
  h_out[3] = p.C;
  h_out[4] = p.max_chunks;
  for (int u = 0; u < p.units; ++u) {
    h_out[5 + 2 * u] = p.W ? pp::plan_cta_of(p, pp::plan_unit_begin(p, u)) : 0;
    h_out[6 + 2 * u] =
        p.W ? pp::plan_cta_of(p, pp::plan_unit_begin(p, u) + pp::plan_unit_tiles(p, u % p.G) - 1)
            : -1;
  }
  return PP_OK;
}

}  // namespace

extern "C" {

#define PP_API __attribute__((visibility("default")))

PP_API const char* pp_status_str(int32_t status) {
  switch (status) {
    case PP_OK: return "PP_OK";
    case PP_ERR_INVALID_ARG: return "PP_ERR_INVALID_ARG";
    case PP_ERR_UNSUPPORTED: return "PP_ERR_UNSUPPORTED";
    case PP_ERR_CAPACITY: return "PP_ERR_CAPACITY";
    case PP_ERR_CUDA: return "PP_ERR_CUDA";
    case PP_ERR_DEVICE_TIMEOUT: return "PP_ERR_DEVICE_TIMEOUT";
    default: return "PP_ERR_UNKNOWN";
  }
}

PP_API int32_t pp_abi_version(void) { return PP_ABI_VERSION; }

PP_API pp_status pp_kv_reset(const pp_kv_layer* layer, void* stream) {
  NvtxRange nvtx_range("pp_kv_reset");
  pp_status s = check_layer(layer);
  if (s != PP_OK) return s;
  return from_cuda(pp::launch_kv_reset(*layer, static_cast<cudaStream_t>(stream)));
}

PP_API pp_status pp_kv_reset_streams(const pp_kv_layer* layer, const int16_t* sid, int32_t n,
                                     void* stream) {
  NvtxRange nvtx_range("pp_kv_reset_streams");
  pp_status s = check_layer(layer);
  if (s != PP_OK) return s;
  if (n < 0) return PP_ERR_INVALID_ARG;
  if (n == 0) return PP_OK;
  if (!sid || !aligned(sid, 2)) return PP_ERR_INVALID_ARG;
  return from_cuda(
      pp::launch_kv_reset_streams(*layer, sid, n, static_cast<cudaStream_t>(stream)));
}

PP_API pp_status pp_kv_append(const pp_kv_layer* layer, const uint16_t* k, const uint16_t* v,
                       const int16_t* sid, const int32_t* pos, int32_t n, void* stream) {
  NvtxRange nvtx_range("pp_kv_append");
  pp_status s = check_layer(layer);
  if (s != PP_OK) return s;
  if (n < 0) return PP_ERR_INVALID_ARG;
  if (n == 0) return PP_OK;
  if (!k || !v || !sid || !pos || !aligned(k, 16) || !aligned(v, 16) || !aligned(sid, 2) ||
      !aligned(pos, 4))
    return PP_ERR_INVALID_ARG;
  return from_cuda(pp::launch_kv_append(*layer, k, v, sid, pos, n, static_cast<cudaStream_t>(stream)));
}

PP_API size_t pp_decode_workspace_bytes(int32_t P, int32_t H, int32_t d, int32_t doc_len,
                                 const pp_options* opt) {
  return workspace(P, H, d, doc_len, opt);
}

PP_API size_t pp_prefill_workspace_bytes(int32_t R, int32_t H, int32_t d, int32_t doc_len,
                                  const pp_options* opt) {
  return workspace(R, H, d, doc_len, opt, false, true);
}

PP_API pp_status pp_decode_attn(const pp_kv_layer* layer, int32_t doc_len, const uint16_t* q,
                         const int16_t* q_sid, const int32_t* q_pos, int32_t P, float scale,
                         uint16_t* o, float* lse, void* ws, size_t ws_bytes, const pp_options* opt,
                         void* stream) {
  NvtxRange nvtx_range("pp_decode_attn");
  if (layer && P > layer->P_max) return PP_ERR_UNSUPPORTED;
  return attend(layer, doc_len, q, q_sid, q_pos, P, scale, o, lse, ws, ws_bytes, opt, stream,
                false, true);
}

PP_API pp_status pp_decode_step(const pp_kv_layer* layer, int32_t doc_len, const uint16_t* k,
                                const uint16_t* v, const uint16_t* q, const int16_t* q_sid,
                                const int32_t* q_pos, int32_t P, float scale, uint16_t* o,
                                float* lse, void* ws, size_t ws_bytes, const pp_options* opt,
                                void* stream) {
  NvtxRange nvtx_range("pp_decode_step");
  if (layer && P > layer->P_max) return PP_ERR_UNSUPPORTED;
  if (P > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16))) return PP_ERR_INVALID_ARG;
  return attend(layer, doc_len, q, q_sid, q_pos, P, scale, o, lse, ws, ws_bytes, opt, stream,
                false, true, k, v);
}

PP_API pp_status pp_prefill_attn(const pp_kv_layer* layer, int32_t doc_len, const uint16_t* q,
                          const int16_t* q_sid, const int32_t* q_pos, int32_t R, float scale,
                          uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                          const pp_options* opt, void* stream) {
  NvtxRange nvtx_range("pp_prefill_attn");
  return attend(layer, doc_len, q, q_sid, q_pos, R, scale, o, lse, ws, ws_bytes, opt, stream);
}

PP_API size_t pp_doc_prefill_workspace_bytes(int32_t H, int32_t d, int32_t doc_len,
                                             const pp_options* opt) {
  return workspace(doc_len, H, d, doc_len, opt, true);
}

PP_API pp_status pp_doc_prefill_attn(const pp_kv_layer* layer, int32_t doc_len, const uint16_t* q,
                                     float scale, uint16_t* o, float* lse, void* ws,
                                     size_t ws_bytes, const pp_options* opt, void* stream) {
  NvtxRange nvtx_range("pp_doc_prefill_attn");
  return attend(layer, doc_len, q, nullptr, nullptr, doc_len, scale, o, lse, ws, ws_bytes, opt,
                stream, true);
}

PP_API pp_status pp_kv8_reset(const pp_kv8_layer* layer, void* stream) {
  NvtxRange nvtx_range("pp_kv8_reset");
  pp_status s = check_kv8_layer(layer);
  if (s != PP_OK) return s;
  return from_cuda(pp::launch_kv8_reset(*layer, static_cast<cudaStream_t>(stream)));
}

PP_API pp_status pp_kv8_append(const pp_kv8_layer* layer, const pp_kv8_append_args* args,
                               void* stream) {
  NvtxRange nvtx_range("pp_kv8_append");
  return kv8_append(layer, args, stream);
}

PP_API size_t pp_kv8_decode_workspace_bytes(int32_t P, int32_t Hq, int32_t H, int32_t d,
                                            int32_t doc_len, const pp_options* opt) {
  return kv8_workspace(P, Hq, H, d, doc_len, opt, true);
}

PP_API size_t pp_kv8_prefill_workspace_bytes(int32_t R, int32_t Hq, int32_t H, int32_t d,
                                             int32_t doc_len, const pp_options* opt) {
  return kv8_workspace(R, Hq, H, d, doc_len, opt, false);
}

PP_API pp_status pp_kv8_decode_attn(const pp_kv8_layer* layer, const pp_kv8_attn_args* args,
                                    void* stream) {
  NvtxRange nvtx_range("pp_kv8_decode_attn");
  return kv8_attend(layer, args, stream, true);
}

PP_API pp_status pp_kv8_prefill_attn(const pp_kv8_layer* layer, const pp_kv8_attn_args* args,
                                     void* stream) {
  NvtxRange nvtx_range("pp_kv8_prefill_attn");
  return kv8_attend(layer, args, stream, false);
}

PP_API pp_status pp_kv8_get_device_status(const pp_kv8_layer* layer, int32_t* h_status,
                                          void* stream) {
  NvtxRange nvtx_range("pp_kv8_get_device_status");
  pp_status s = check_kv8_layer(layer);
  if (s != PP_OK) return s;
  if (!h_status) return PP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(h_status, layer->status, sizeof(int32_t), cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return PP_ERR_CUDA;
  if ((s = from_cuda(cudaStreamSynchronize(st))) != PP_OK) return s;
  return (*h_status & PP_DEV_TIMEOUT) ? PP_ERR_DEVICE_TIMEOUT : PP_OK;
}

PP_API pp_status pp_debug_visibility(const pp_kv_layer* layer, int32_t doc_len, const int16_t* q_sid,
                              const int32_t* q_pos, int32_t nq, int32_t* count_out,
                              uint8_t* mask_out, void* stream) {
  pp_status s = check_layer(layer);
  if (s != PP_OK) return s;
  if (nq < 0 || doc_len < 0) return PP_ERR_INVALID_ARG;
  if (doc_len > layer->doc_cap) return PP_ERR_CAPACITY;
  if (nq == 0) return PP_OK;
  if (!q_sid || !q_pos || !count_out) return PP_ERR_INVALID_ARG;
  return from_cuda(pp::launch_visibility(*layer, doc_len, q_sid, q_pos, nq, count_out, mask_out,
                                         static_cast<cudaStream_t>(stream)));
}

PP_API pp_status pp_debug_split_plan(int32_t rows, int32_t H, int32_t doc_len, int32_t ctas,
                              int64_t* h_out, int32_t h_out_len) {
  if (rows < 0 || H < 1 || doc_len < 0 || ctas < 1 || !h_out) return PP_ERR_INVALID_ARG;
  return write_plan(make_plan(rows, H, doc_len, ctas), h_out, h_out_len);
}

PP_API pp_status pp_debug_split_plan_causal(int32_t doc_len, int32_t H, int32_t ctas,
                                            int64_t* h_out, int32_t h_out_len) {
  if (H < 1 || doc_len < 0 || ctas < 1 || !h_out) return PP_ERR_INVALID_ARG;
  return write_plan(make_plan(doc_len, H, doc_len, ctas, true), h_out, h_out_len);
}

PP_API pp_status pp_debug_kv8_runs(int32_t rows, int32_t Hq, int32_t H, int32_t doc_len,
                                   int32_t decode, int32_t splits, int32_t num_sms, int64_t* h_out,
                                   int32_t h_out_len) {
  if (rows < 0 || H < 1 || Hq < 1 || Hq % H != 0 || doc_len < 0 || splits < 0 || num_sms < 1 ||
      !h_out)
    return PP_ERR_INVALID_ARG;
  if ((int64_t)rows * Hq > INT32_MAX - 256) return PP_ERR_UNSUPPORTED;
  pp_options opt{};
  opt.splits = splits;
  const SplitPlan p = kv8_plan(rows, Hq, H, doc_len, &opt, decode != 0, num_sms);
  if (p.W > INT32_MAX) return PP_ERR_UNSUPPORTED;
  return write_kv8_runs(p, rows * (Hq / H), pp::kv8_items(rows, Hq / H, H, decode != 0), h_out,
                        h_out_len);
}

PP_API pp_status pp_debug_exp2(const float* x, float* y_poly, float* y_hw, int32_t n,
                               void* stream) {
  if (n < 0) return PP_ERR_INVALID_ARG;
  if (n == 0) return PP_OK;
  if (!x || !y_poly || !y_hw || !aligned(x, 4) || !aligned(y_poly, 4) || !aligned(y_hw, 4))
    return PP_ERR_INVALID_ARG;
  return from_cuda(pp::launch_exp2(x, y_poly, y_hw, n, static_cast<cudaStream_t>(stream)));
}

PP_API pp_status pp_get_device_status(const pp_kv_layer* layer, int32_t* h_status, void* stream) {
  NvtxRange nvtx_range("pp_get_device_status");
  pp_status s = check_layer(layer);
  if (s != PP_OK) return s;
  if (!h_status) return PP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(h_status, layer->status, sizeof(int32_t), cudaMemcpyDeviceToHost, st) !=
      cudaSuccess)
    return PP_ERR_CUDA;
  if ((s = from_cuda(cudaStreamSynchronize(st))) != PP_OK) return s;
  return (*h_status & PP_DEV_TIMEOUT) ? PP_ERR_DEVICE_TIMEOUT : PP_OK;
}

}  // extern "C"
