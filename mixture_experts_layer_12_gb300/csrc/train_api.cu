// train_api.cu -- the C ABI declared in include/moe_train.h: argument checks,
// workspace layouts, tensor maps and the launches of each call on the caller's
// stream.  No allocation and no host synchronisation.
#include <initializer_list>
#include <mutex>

#include "api_internal.h"
#include "moe_train.h"
#include "train_internal.h"

using namespace moe;

namespace {

std::mutex g_mu;
bool g_ready[kMaxDevices];

// device_setup() and, on a device's first use here, the attributes of these
// kernels (callers of the other entry points do not load them).
int train_setup(int* sms) {
  int rc = device_setup(sms);
  if (rc != MOE_OK) return rc;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_ready[dev]) {
    if ((e = train_gemm_set_attributes()) != cudaSuccess) return cuda_fail(e, "training attributes");
    g_ready[dev] = true;
  }
  return MOE_OK;
}

#define CUDA_TRY(call, what)                          \
  do {                                                \
    const cudaError_t err_ = (call);                  \
    if (err_ != cudaSuccess) return cuda_fail(err_, what); \
  } while (0)
#define TRY(call)                 \
  do {                            \
    const int rc_ = (call);       \
    if (rc_ != MOE_OK) return rc_; \
  } while (0)

size_t up(size_t v) { return (v + 1023) / 1024 * 1024; }

bool gated(const moe_shape* s) { return s->expert_act == MOE_EXPERT_SWIGLU; }
int halves(const moe_shape* s) { return gated(s) ? 2 : 1; }
size_t rows_of(const moe_shape* s) { return (size_t)s->T * s->k; }
int ep_of(const moe_shape* s) { return (s->E + 7) / 8 * 8; }
size_t pad_of(const moe_shape* s) { return padded_rows_cap(rows_of(s), s->E); }

// Regions of a workspace, handed out one after the other.
struct Carve {
  char* base;
  size_t used = 0;
  explicit Carve(void* p) : base(static_cast<char*>(p)) {}
  template <typename T>
  T* take(size_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += up(n * sizeof(T));
    return p;
  }
};

// Rows of a workspace matrix start on 128 bytes: TMA boxes of 128-byte rows then
// read 4 sectors of one line, not 5 of two (8000 rows, 8 experts of 2872 x 9480:
// a weight gradient 367 us against 306 with 2880 x 9472, which need none of this).
size_t ld_of(size_t cols) { return (cols + 63) / 64 * 64; }

// [rows, cols] bf16, rows `ld` columns apart
int map_rows(CUtensorMap* m, const void* base, size_t cols, size_t ld, size_t rows, uint32_t box_rows,
             const char* what) {
  const uint64_t dims[2] = {cols, rows};
  const uint64_t strides[1] = {ld * 2};
  const uint32_t box[2] = {64, box_rows};
  return encode_map_as(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, 2, dims, strides, box,
                       what);
}
int map_weights(CUtensorMap* m, const void* base, size_t cols, size_t rows, size_t n, uint32_t box_rows,
                const char* what) {
  const uint64_t dims[3] = {cols, rows, n};
  const uint64_t strides[2] = {cols * 2, cols * rows * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_map_as(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, 3, dims, strides, box,
                       what);
}
// Output [n, rows, cols] of a weight gradient.
int map_out(CUtensorMap* m, const void* base, size_t cols, size_t rows, size_t n, bool f32) {
  const uint64_t size = f32 ? 4 : 2;
  const uint64_t dims[3] = {cols, rows, n};
  const uint64_t strides[2] = {cols * size, cols * rows * size};
  const uint32_t box[3] = {(uint32_t)(64 / size), 32, 1};
  return encode_map_as(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       CU_TENSOR_MAP_SWIZZLE_64B, base, 3, dims, strides, box, "weight gradient");
}

SegArgs segments(const moe_shape* s, const int32_t* offsets) {
  SegArgs g;
  g.offsets = offsets;
  g.E = s->E;
  g.rows = (int)rows_of(s);
  g.rows_pad = (int)pad_of(s);
  g.chunk = 0;
  return g;
}
// `rows` rows in chunks of `chunk`, not padded
SegArgs chunks(int rows, int chunk) {
  SegArgs g;
  g.offsets = nullptr;
  g.E = (rows + chunk - 1) / chunk;
  g.rows = rows;
  g.rows_pad = (rows + kSegPad - 1) / kSegPad * kSegPad;
  g.chunk = chunk;
  return g;
}
TrainGemmArgs gemm_args(const SegArgs& seg, int M, int N, int K, void* status) {
  TrainGemmArgs a = {};
  a.seg = seg;
  a.M = M;
  a.N = N;
  a.K = K;
  a.splits = 1;
  a.ksplit = (K + 63) / 64;
  a.status = static_cast<int*>(status);
  a.wait_limit_ns = kWaitLimitNs;
  return a;
}
int64_t row_tiles(size_t rows, int E, int cols, int per) {
  return (int64_t)((rows + 255) / 256 + (rows < (size_t)E ? rows : (size_t)E)) * ((cols + per - 1) / per);
}
int64_t blocks256(int n) { return ((int64_t)n + 255) / 256; }

// CTA pairs that plans count on: one per two of the part's 152 SMs.  A number and
// not the device's count, so that workspace sizes, which are asked for without a
// device, and the order of sums depend on the shape alone; where fewer pairs are
// resident, what was planned as one round of tiles takes two.
constexpr int kPlanPairs = 76;

// Parts of K for a product whose fp32 outputs are summed afterwards anyway: few
// rows leave most CTA pairs without a tile, and a long K then takes its time on a
// few of them (3 rows of 3 experts of 576 x 14096: 73 us).  At most `most` parts of
// at least `least` stages, and together no more tiles than pairs.
struct Split {
  int parts, stages;
};
Split split_of(int64_t blocks, int cols, int K, int most, int least) {
  const int kb = (K + 63) / 64;
  const int64_t tiles = blocks * ((cols + 255) / 256);
  int64_t S = tiles > 0 ? kPlanPairs / tiles : 1;
  if (S > most) S = most;
  if (S > kb / least) S = kb / least;
  if (S < 1) S = 1;
  Split p;
  p.stages = (int)((kb + S - 1) / S);
  p.parts = (kb + p.stages - 1) / p.stages;
  return p;
}
// Products whose rows are summed by token: 8 parts of 8 stages or more (the sum
// reads every part).
Split row_split(size_t rows, int E, int cols, int K) {
  const int64_t n = (int64_t)rows, hit = n < E ? n : E;
  return split_of(hit > 0 ? hit * (((n + hit - 1) / hit + 255) / 256) : 0, cols, K, 8, 8);
}

// ------------------------------------------------------------------ products --

int fwd_product(const moe_shape* s, int bits, const uint16_t* xp, size_t ld_xp, const uint16_t* w1, const int32_t* offsets,
                uint16_t* h, void* z, uint8_t* z_scales, const int* merge, void* status, cudaStream_t st) {
  const size_t rows = rows_of(s);
  CUtensorMap ta, tb, ta64;
  TRY(map_rows(&ta, xp, s->H, ld_xp, rows, 128, "xp"));
  TRY(map_rows(&ta64, xp, s->H, ld_xp, rows, 64, "xp"));
  TRY(map_weights(&tb, w1, (size_t)s->F * halves(s), s->H, s->E, 64, "W1"));
  TrainGemmArgs a = gemm_args(segments(s, offsets), 0, s->F, s->H, status);
  a.out = h;
  a.ld_out = (int)ld_of(s->F);
  a.keep_bits = bits;
  a.z = z;
  a.z_scales = z_scales;
  a.merge_status = merge;
  CUDA_TRY(launch_train_gemm(gated(s) ? kTrainFwdSwiGLU : kTrainFwdGelu, ta, tb, ta64, a,
                             row_tiles(rows, s->E, s->F, gated(s) ? 128 : 256), st),
           "expert GEMM1 launch");
  return MOE_OK;
}

// Y = h W2 in bf16, or (Y32) in fp32
int plain_product(const moe_shape* s, const uint16_t* h, const uint16_t* w2, const int32_t* offsets, uint16_t* Y,
                  float* Y32, void* status, cudaStream_t st) {
  const size_t rows = rows_of(s);
  CUtensorMap ta, tb, ta64;
  TRY(map_rows(&ta, h, s->F, ld_of(s->F), rows, 128, "h"));
  TRY(map_rows(&ta64, h, s->F, ld_of(s->F), rows, 64, "h"));
  TRY(map_weights(&tb, w2, s->H, s->F, s->E, 64, "W2"));
  TrainGemmArgs a = gemm_args(segments(s, offsets), 0, s->H, s->F, status);
  a.out = Y;
  a.ld_out = s->H;
  a.out32 = Y32;
  if (Y32) {  // (bf16 outputs are rounded at once: K in one part)
    const Split sp = row_split(rows, s->E, s->H, s->F);
    a.splits = sp.parts;
    a.ksplit = sp.stages;
  }
  CUDA_TRY(launch_train_gemm(Y32 ? kTrainPlain : kTrainPlainBf16, ta, tb, ta64, a,
                             row_tiles(rows, s->E, s->H, 256) * a.splits, st),
           "expert GEMM2 launch");
  return MOE_OK;
}

// The experts' gradients from padded xp and dyp; dxp compact, in bf16 or (dxp
// null) as the parts of row_split in dxp32.
struct FfnGrad {
  int bits;
  const uint16_t *xp, *dyp, *w1, *w2;
  const int32_t* offsets;
  const void* z;
  const uint8_t* z_scales;
  const float* w;
  const int32_t* perm;
  float* part;
  uint16_t *hw, *dz, *dxp, *dw1, *dw2;
  float* dxp32;
};
int ffn_gradients(const moe_shape* s, const FfnGrad& f, void* status, cudaStream_t st) {
  const size_t rows = rows_of(s), pad = pad_of(s);
  const int f1 = s->F * halves(s);
  const SegArgs seg = segments(s, f.offsets);
  CUtensorMap ta, tb, ta64;
  // g = dy W2^T; dz, w h, <g, h>
  TRY(map_rows(&ta, f.dyp, s->H, ld_of(s->H), pad, 128, "dy rows"));
  TRY(map_rows(&ta64, f.dyp, s->H, ld_of(s->H), pad, 64, "dy rows"));
  TRY(map_weights(&tb, f.w2, s->H, s->F, s->E, 128, "W2"));
  TrainGemmArgs a = gemm_args(seg, 0, s->F, s->H, status);
  a.keep_bits = f.bits;
  a.z = const_cast<void*>(f.z);
  a.z_scales = const_cast<uint8_t*>(f.z_scales);
  a.w = f.w;
  a.perm = f.perm;
  a.n_w = (int)rows;
  a.dz = f.dz;
  a.hw = f.hw;
  a.ld_dz = (int)ld_of(f1);
  a.ld_hw = (int)ld_of(s->F);
  a.part = f.part;
  a.units = (s->F + 63) / 64;
  CUDA_TRY(launch_train_gemm(gated(s) ? kTrainBwdSwiGLU : kTrainBwdGelu, ta, tb, ta64, a,
                             row_tiles(rows, s->E, s->F, 256), st),
           "h gradient launch");
  // dW2 = (w h)^T dy
  TRY(map_rows(&ta, f.hw, s->F, ld_of(s->F), pad, 64, "w h"));
  TRY(map_rows(&tb, f.dyp, s->H, ld_of(s->H), pad, 64, "dy rows"));
  a = gemm_args(seg, s->F, s->H, 0, status);
  a.out = f.dw2;
  TRY(map_out(&ta64, f.dw2, s->H, s->F, s->E, false));
  CUDA_TRY(launch_train_gemm(kTrainWgrad, ta, tb, ta64, a, s->E * blocks256(s->F) * blocks256(s->H), st),
           "dW2 launch");
  // dW1 = xp^T dz
  TRY(map_rows(&ta, f.xp, s->H, ld_of(s->H), pad, 64, "xp"));
  TRY(map_rows(&tb, f.dz, f1, ld_of(f1), pad, 64, "dz"));
  a = gemm_args(seg, s->H, f1, 0, status);
  a.out = f.dw1;
  TRY(map_out(&ta64, f.dw1, f1, s->H, s->E, false));
  CUDA_TRY(launch_train_gemm(kTrainWgrad, ta, tb, ta64, a, s->E * blocks256(s->H) * blocks256(f1), st),
           "dW1 launch");
  // dxp = dz W1^T
  TRY(map_rows(&ta, f.dz, f1, ld_of(f1), pad, 128, "dz"));
  TRY(map_rows(&ta64, f.dz, f1, ld_of(f1), pad, 64, "dz"));
  TRY(map_weights(&tb, f.w1, f1, s->H, s->E, 128, "W1"));
  a = gemm_args(seg, 0, s->H, f1, status);
  a.out = f.dxp;
  a.ld_out = s->H;
  a.out32 = f.dxp32;
  const Split sp = row_split(rows, s->E, s->H, f1);
  a.splits = sp.parts;
  a.ksplit = sp.stages;
  // (rounded at once where K is not split and nobody sums the rows)
  const bool f32 = sp.parts > 1 || !f.dxp;
  CUDA_TRY(launch_train_gemm(f32 ? kTrainRowsF32 : kTrainRows, ta, tb, ta64, a,
                             row_tiles(rows, s->E, s->H, 256) * (f32 ? sp.parts : 1), st),
           "x gradient launch");
  if (f32 && f.dxp) {
    RowsSumArgs sum = {};
    sum.rows32 = f.dxp32;
    sum.splits = sp.parts;
    sum.range = f.offsets;
    sum.E = s->E;
    sum.T = (int)rows;
    sum.H = s->H;
    sum.k = 1;
    sum.out = f.dxp;
    CUDA_TRY(launch_rows_sum(sum, st), "x gradient sums launch");
  }
  return MOE_OK;
}

// Splits of the router's weight gradient along the tokens: as many as give every
// CTA pair a tile, but at least 256 tokens each (its fp32 partial outputs are
// written and read again).
int router_chunk(const moe_shape* s) {
  const int64_t tiles = blocks256(s->H) * blocks256(2 * ep_of(s));
  int64_t S = kPlanPairs / tiles;
  if (S > s->T / 256) S = s->T / 256;
  if (S < 1) S = 1;
  if (S > kMaxExperts) S = kMaxExperts;
  const int64_t c = (s->T + S - 1) / S;
  return (int)((c + 63) / 64 * 64);
}
int router_splits(const moe_shape* s) {
  const int c = router_chunk(s);
  return (s->T + c - 1) / c;
}

struct RouteGradWs {
  uint16_t *dl, *w;
  float *part, *db_part, *dlk;
};
RouteGradWs route_grad_ws(const moe_shape* s, Carve& c) {
  const size_t ep2 = 2 * (size_t)ep_of(s);
  RouteGradWs r;
  r.dl = c.take<uint16_t>(s->T * ep2);
  r.w = c.take<uint16_t>(s->H * ep2);
  r.dlk = c.take<float>(rows_of(s));
  r.part = c.take<float>(s->T > 0 ? router_splits(s) * (size_t)s->H * ep2 : 0);
  r.db_part = c.take<float>((size_t)((s->T + kGateTokens - 1) / kGateTokens) * s->E);
  return r;
}
// Whether dx's router part is a product over all experts: with a softmax over all
// every expert has one; else only a token's k chosen ones, which the sum over its
// rows takes along while they are few (2048 tokens of 4096 columns, k = 8: 22 us,
// 12 as a product; 8192 of 2048, k = 4, with the rows: see rows_sum_kernel).
bool router_product(const moe_shape* s) { return s->gating == MOE_GATE_SOFTMAX_TOPK || s->k > 4; }

// dW_router, db and dx, whose other parts `sum` has; the router's as a product
// goes into dx, or in fp32 into `add`.
int route_gradients(const moe_shape* s, const RouteGradWs& r, const GateBackwardArgs& gate, const uint16_t* x,
                    uint16_t* dw_router, float* db, float* add, RowsSumArgs sum, void* status, cudaStream_t st) {
  const int ep = ep_of(s);
  CUDA_TRY(launch_gate_backward(gate, st), "gate gradient launch");
  CUtensorMap ta, tb, ta64;
  // dW_router's partial sums = x^T dlogits over chunks of tokens
  TRY(map_rows(&ta, x, s->H, s->H, s->T, 64, "x"));
  TRY(map_rows(&tb, r.dl, 2 * ep, 2 * ep, s->T, 64, "dlogits"));
  TrainGemmArgs a = gemm_args(chunks(s->T, router_chunk(s)), s->H, 2 * ep, 0, status);
  a.out32 = r.part;
  TRY(map_out(&ta64, r.part, 2 * ep, s->H, a.seg.E, true));
  CUDA_TRY(launch_train_gemm(kTrainWgradF32, ta, tb, ta64, a, a.seg.E * blocks256(s->H) * blocks256(2 * ep), st),
           "dW_router launch");
  RouterReduceArgs ra;
  ra.H = s->H;
  ra.E = s->E;
  ra.ep = ep;
  ra.S = a.seg.E;
  ra.part = r.part;
  ra.dw_router = dw_router;
  ra.db_part = r.db_part;
  ra.n_db = (s->T + kGateTokens - 1) / kGateTokens;
  ra.db = db;
  CUDA_TRY(launch_router_reduce(ra, st), "dW_router sums launch");
  if (router_product(s)) {
    TRY(map_rows(&ta, r.dl, 2 * ep, 2 * ep, s->T, 128, "dlogits"));
    TRY(map_rows(&ta64, r.dl, 2 * ep, 2 * ep, s->T, 64, "dlogits"));
    TRY(map_weights(&tb, r.w, 2 * ep, s->H, 1, 128, "W_router"));
    a = gemm_args(chunks(s->T, (s->T + kSegPad - 1) / kSegPad * kSegPad), 0, s->H, 2 * ep, status);
    a.out = sum.out;
    a.ld_out = s->H;
    a.out32 = add;
    CUDA_TRY(launch_train_gemm(add ? kTrainRowsF32 : kTrainRows, ta, tb, ta64, a,
                               blocks256(s->T) * blocks256(s->H), st),
             "router x gradient launch");
    if (!add) return MOE_OK;
    sum.add = add;
  } else {
    sum.dl = r.dlk;
    sum.ids = gate.ids;
    sum.wt = r.w;
    sum.E = s->E;
  }
  CUDA_TRY(launch_rows_sum(sum, st), "row sums launch");
  return MOE_OK;
}
GateBackwardArgs gate_args(const moe_shape* s, const RouteGradWs& r, const uint16_t* w_router, const int32_t* ids,
                           const float* weights, const float* probs) {
  GateBackwardArgs g = {};
  g.T = s->T;
  g.E = s->E;
  g.k = s->k;
  g.ep = ep_of(s);
  g.gating = s->gating;
  g.ids = ids;
  g.weights = weights;
  g.probs = probs;
  g.dl = r.dl;
  g.db_part = r.db_part;
  g.w_router = w_router;
  g.H = s->H;
  if (router_product(s)) {
    g.w2 = r.w;
  } else {
    g.wt = r.w;
    g.dlk = r.dlk;
  }
  return g;
}

// The router's logits, few columns: up to 64 parts of 4 stages or more (one wave
// of 8 tiles with K = 4096 took 28 us, 11 in parts).
Split probs_split(const moe_shape* s) {
  return split_of(blocks256(s->T), ep_of(s), s->H, 64, 4);
}

struct ProbsWs {
  uint16_t* wpad;
  float* logits;
};
ProbsWs probs_ws(const moe_shape* s, Carve& c) {
  ProbsWs p;
  p.wpad = c.take<uint16_t>(s->E % 8 ? (size_t)s->H * ep_of(s) : 0);
  p.logits = c.take<float>(probs_split(s).parts * (size_t)s->T * ep_of(s));
  return p;
}
int router_probs(const moe_shape* s, int sms, const ProbsWs& p, const uint16_t* x, const uint16_t* w_router,
                 const float* b_router, float* probs, void* status, cudaStream_t st) {
  const int ep = ep_of(s);
  if (s->E % 8) {
    CUDA_TRY(launch_pad_router_weights(w_router, s->H, s->E, ep, p.wpad, sms, st, true),
             "router weight padding launch");
    w_router = p.wpad;
  }
  CUtensorMap ta, tb, ta64;
  TRY(map_rows(&ta, x, s->H, s->H, s->T, 128, "x"));
  TRY(map_rows(&ta64, x, s->H, s->H, s->T, 64, "x"));
  TRY(map_weights(&tb, w_router, ep, s->H, 1, 64, "W_router"));
  const Split sp = probs_split(s);
  TrainGemmArgs a = gemm_args(chunks(s->T, (s->T + kSegPad - 1) / kSegPad * kSegPad), 0, ep, s->H, status);
  a.out32 = p.logits;
  a.splits = sp.parts;
  a.ksplit = sp.stages;
  CUDA_TRY(launch_train_gemm(kTrainPlain, ta, tb, ta64, a, sp.parts * blocks256(s->T) * blocks256(ep), st),
           "router logits launch");
  CUDA_TRY(launch_router_softmax(p.logits, sp.parts, ep, b_router, s->T, s->E, probs, st), "router softmax launch");
  return MOE_OK;
}

// ---------------------------------------------------------------- workspaces --

struct FfnWs {
  uint16_t* h;
};
FfnWs ffn_ws(const moe_shape* s, Carve& c) {
  FfnWs w;
  w.h = c.take<uint16_t>(rows_of(s) * ld_of(s->F));
  return w;
}

struct FfnGradWs {
  uint16_t *xp, *dyp, *hw, *dz;
  float* dxp;  // parts of row_split
};
// layer: dxp is summed by token, in fp32 in any case
FfnGradWs ffn_grad_ws(const moe_shape* s, bool layer, Carve& c) {
  const size_t pad = pad_of(s);
  FfnGradWs w;
  w.xp = c.take<uint16_t>(pad * ld_of(s->H));
  w.dyp = c.take<uint16_t>(pad * ld_of(s->H));
  w.hw = c.take<uint16_t>(pad * ld_of(s->F));
  w.dz = c.take<uint16_t>(pad * ld_of((size_t)s->F * halves(s)));
  const int parts = row_split(rows_of(s), s->E, s->H, s->F * halves(s)).parts;
  w.dxp = c.take<float>(parts > 1 || layer ? parts * rows_of(s) * s->H : 0);
  return w;
}

struct ForwardWs {
  void* route;
  size_t route_bytes;
  uint16_t* xp;
  float* Y;
  FfnWs ffn;
  ProbsWs probs;
};
ForwardWs forward_ws(const moe_shape* s, Carve& c) {
  ForwardWs w = {};
  w.route_bytes = moe_route_workspace_size(s);
  w.route = c.take<char>(w.route_bytes);
  // xp and, once it has been read, the experts' outputs in row_split's parts
  const size_t y = row_split(rows_of(s), s->E, s->H, s->F).parts * (size_t)s->H, x = (ld_of(s->H) + 1) / 2;
  w.Y = c.take<float>(rows_of(s) * (y > x ? y : x));
  w.xp = reinterpret_cast<uint16_t*>(w.Y);  // read before Y is written
  w.ffn = ffn_ws(s, c);
  if (s->gating == MOE_GATE_SOFTMAX_TOPK) w.probs = probs_ws(s, c);
  return w;
}

struct BackwardWs {
  FfnGradWs ffn;
  uint16_t* x;  // bf16 of x kept in 8 bits
  float* part;
  RouteGradWs route;
  float* dxr;  // the router's part of dx
};
BackwardWs backward_ws(const moe_shape* s, int bits, Carve& c) {
  BackwardWs w;
  w.ffn = ffn_grad_ws(s, true, c);
  w.x = c.take<uint16_t>(bits == 8 ? (size_t)s->T * s->H : 0);
  w.part = c.take<float>(rows_of(s) * ((s->F + 63) / 64));
  w.route = route_grad_ws(s, c);
  w.dxr = c.take<float>(router_product(s) ? (size_t)s->T * s->H : 0);
  return w;
}

// moe.h's limits, and below the sizes whose grids (row sums: 1024 columns a block
// of y, at most 65535) or numbers of columns (2 F) would not fit.
int check_train_shape(const moe_shape* s, bool need_ffn) {
  TRY(check_shape(s, need_ffn));
  if (s->H > 1 << 25) return fail(MOE_ERR_UNSUPPORTED, "H = %d: at most 2^25", s->H);
  if (need_ffn && s->F > 1 << 29) return fail(MOE_ERR_UNSUPPORTED, "F = %d: at most 2^29", s->F);
  return MOE_OK;
}

int check_bits(int32_t bits) {
  if (bits != 8 && bits != 16) return fail(MOE_ERR_INVALID_ARG, "keep_bits = %d: 8 or 16", bits);
  return MOE_OK;
}

#define CHECK_WS(need, name)                                                                        \
  do {                                                                                              \
    REQUIRE_PTR(status);                                                                            \
    REQUIRE_PTR(ws);                                                                                \
    if (ws_bytes < (need))                                                                          \
      return fail(MOE_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed (%s)", ws_bytes, (size_t)(need), \
                  name);                                                                            \
  } while (0)

// The bytes that a call reads or writes of a buffer (null: none).
struct Span {
  const void* p;
  size_t bytes;
  const char* name;
};
#define SPAN(p, n) Span{p, (size_t)(n) * sizeof(*(p)), #p}

// What a call writes lies apart from what it reads and from the rest of what it
// writes: blocks finish in any order, some while others still read.
int check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  const auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
  };
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (meet(*o, i)) return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (meet(*o, *q)) return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
  }
  return MOE_OK;
}
// Elements of the experts' weights, of kept z and of its scales.
size_t w1_of(const moe_shape* s) { return (size_t)s->E * s->H * s->F * halves(s); }
size_t w2_of(const moe_shape* s) { return (size_t)s->E * s->F * s->H; }
Span kept_span(const moe_shape* s, int bits, const void* z) {
  return Span{z, rows_of(s) * halves(s) * s->F * (bits / 8), "z"};
}
Span kept_scales_span(const moe_shape* s, int bits, const uint8_t* z_scales) {
  return Span{z_scales, bits == 8 ? rows_of(s) * halves(s) * (((size_t)s->F + 31) / 32) : 0, "z_scales"};
}

int check_a8(int64_t rows, int32_t cols) {
  if (rows < 0 || cols < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %lld, cols = %d", (long long)rows, cols);
  if (cols < 8 || cols % 8) return fail(MOE_ERR_UNSUPPORTED, "cols = %d: need cols >= 8, cols %% 8 == 0", cols);
  if (rows >= ((int64_t)1 << 46) / cols)
    return fail(MOE_ERR_UNSUPPORTED, "rows * cols = %lld * %d: need less than 2^46", (long long)rows, cols);
  return MOE_OK;
}

cudaStream_t stream_of(void* s) { return static_cast<cudaStream_t>(s); }

int zero(void* p, size_t bytes, cudaStream_t st) {
  CUDA_TRY(cudaMemsetAsync(p, 0, bytes, st), "cudaMemsetAsync");
  return MOE_OK;
}
int zero_weights(const moe_shape* s, uint16_t* dw1, uint16_t* dw2, cudaStream_t st) {
  const size_t n = (size_t)s->E * s->H * s->F * 2;
  TRY(zero(dw1, n * halves(s), st));
  return zero(dw2, n, st);
}

}  // namespace

// =================================================================== C ABI

extern "C" {

int moet_quantize_a8(int64_t rows, int32_t cols, const uint16_t* x, int8_t* codes, uint8_t* scales,
                     void* stream) {
  TRY(check_a8(rows, cols));
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  const size_t n = (size_t)rows * cols, groups = (size_t)rows * (((size_t)cols + 31) / 32);
  TRY(check_apart({SPAN(codes, n), SPAN(scales, groups)}, {SPAN(x, n)}));
  int sms = 0;
  TRY(device_setup(&sms));
  CUDA_TRY(launch_quantize_a8(rows, cols, x, codes, scales, sms, stream_of(stream)), "quantize launch");
  return MOE_OK;
}

int moet_dequantize_a8(int64_t rows, int32_t cols, const int8_t* codes, const uint8_t* scales, uint16_t* out,
                       void* stream) {
  TRY(check_a8(rows, cols));
  if (rows == 0) return MOE_OK;
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  REQUIRE_PTR(out);
  const size_t n = (size_t)rows * cols, groups = (size_t)rows * (((size_t)cols + 31) / 32);
  TRY(check_apart({SPAN(out, n)}, {SPAN(codes, n), SPAN(scales, groups)}));
  int sms = 0;
  TRY(device_setup(&sms));
  CUDA_TRY(launch_dequantize_a8(rows, cols, codes, scales, out, sms, stream_of(stream)), "dequantize launch");
  return MOE_OK;
}

int moet_dispatch_rows_backward(const moe_shape* s, const uint16_t* dxp, const int32_t* slot, uint16_t* dx,
                                void* stream) {
  TRY(check_train_shape(s, false));
  if (s->T == 0) return MOE_OK;
  REQUIRE_PTR(dxp);
  REQUIRE_PTR(slot);
  REQUIRE_PTR(dx);
  const size_t n = rows_of(s);
  TRY(check_apart({SPAN(dx, (size_t)s->T * s->H)}, {SPAN(dxp, n * s->H), SPAN(slot, n)}));
  int sms = 0;
  TRY(device_setup(&sms));
  RowsSumArgs a = {};
  a.rows = dxp;
  a.slot = slot;
  a.T = s->T;
  a.H = s->H;
  a.k = s->k;
  a.out = dx;
  CUDA_TRY(launch_rows_sum(a, stream_of(stream)), "row sums launch");
  return MOE_OK;
}

int moet_combine_backward(const moe_shape* s, const uint16_t* dy, const uint16_t* Y, const float* weights,
                          const int32_t* slot, uint16_t* dY, float* dweights, void* stream) {
  TRY(check_train_shape(s, false));
  if (s->T == 0) return MOE_OK;
  REQUIRE_PTR(dy);
  REQUIRE_PTR(Y);
  REQUIRE_PTR(weights);
  REQUIRE_PTR(slot);
  REQUIRE_PTR(dY);
  REQUIRE_PTR(dweights);
  const size_t n = rows_of(s);
  TRY(check_apart({SPAN(dY, n * s->H), SPAN(dweights, n)},
                  {SPAN(dy, (size_t)s->T * s->H), SPAN(Y, n * s->H), SPAN(weights, n), SPAN(slot, n)}));
  int sms = 0;
  TRY(device_setup(&sms));
  CombineBackwardArgs a = {dy, Y, weights, slot, s->T, s->H, s->k, dY, dweights};
  CUDA_TRY(launch_combine_backward(a, stream_of(stream)), "combine gradient launch");
  return MOE_OK;
}

size_t moet_expert_ffn_workspace_size(const moe_shape* s) {
  if (check_train_shape(s, true) != MOE_OK) return 0;
  Carve c(nullptr);
  ffn_ws(s, c);
  return c.used + 1024;
}

int moet_expert_ffn(const moe_shape* s, int32_t keep_bits, const uint16_t* xp, const uint16_t* w1,
                    const uint16_t* w2, const int32_t* offsets, uint16_t* Y, void* z, uint8_t* z_scales,
                    void* status, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_train_shape(s, true));
  TRY(check_bits(keep_bits));
  CHECK_WS(moet_expert_ffn_workspace_size(s), "moet_expert_ffn_workspace_size");
  if (s->T == 0) return MOE_OK;
  REQUIRE_PTR(xp);
  REQUIRE_PTR(w1);
  REQUIRE_PTR(w2);
  REQUIRE_PTR(offsets);
  REQUIRE_PTR(Y);
  REQUIRE_PTR(z);
  if (keep_bits == 8) REQUIRE_PTR(z_scales);
  const size_t n = rows_of(s);
  TRY(check_apart({SPAN(Y, n * s->H), kept_span(s, keep_bits, z), kept_scales_span(s, keep_bits, z_scales),
                   Span{status, MOE_WS_MIN_BYTES, "status"}, Span{ws, moet_expert_ffn_workspace_size(s), "ws"}},
                  {SPAN(xp, n * s->H), SPAN(w1, w1_of(s)), SPAN(w2, w2_of(s)), SPAN(offsets, s->E + 1)}));
  int sms = 0;
  TRY(train_setup(&sms));
  Carve c(ws);
  const FfnWs w = ffn_ws(s, c);
  TRY(fwd_product(s, keep_bits, xp, s->H, w1, offsets, w.h, z, z_scales, nullptr, status, stream_of(stream)));
  return plain_product(s, w.h, w2, offsets, Y, nullptr, status, stream_of(stream));
}

size_t moet_expert_ffn_backward_workspace_size(const moe_shape* s) {
  if (check_train_shape(s, true) != MOE_OK) return 0;
  Carve c(nullptr);
  ffn_grad_ws(s, false, c);
  return c.used + 1024;
}

int moet_expert_ffn_backward(const moe_shape* s, int32_t keep_bits, const uint16_t* xp, const void* z,
                             const uint8_t* z_scales, const uint16_t* w1, const uint16_t* w2,
                             const int32_t* offsets, const uint16_t* dY, uint16_t* dxp, uint16_t* dw1,
                             uint16_t* dw2, void* status, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_train_shape(s, true));
  TRY(check_bits(keep_bits));
  CHECK_WS(moet_expert_ffn_backward_workspace_size(s), "moet_expert_ffn_backward_workspace_size");
  REQUIRE_PTR(dw1);
  REQUIRE_PTR(dw2);
  if (s->T > 0) {
    REQUIRE_PTR(xp);
    REQUIRE_PTR(z);
    if (keep_bits == 8) REQUIRE_PTR(z_scales);
    REQUIRE_PTR(w1);
    REQUIRE_PTR(w2);
    REQUIRE_PTR(offsets);
    REQUIRE_PTR(dY);
    REQUIRE_PTR(dxp);
    const size_t n = rows_of(s);
    TRY(check_apart({SPAN(dxp, n * s->H), SPAN(dw1, w1_of(s)), SPAN(dw2, w2_of(s)),
                     Span{status, MOE_WS_MIN_BYTES, "status"}, Span{ws, moet_expert_ffn_backward_workspace_size(s), "ws"}},
                    {SPAN(xp, n * s->H), kept_span(s, keep_bits, z), kept_scales_span(s, keep_bits, z_scales),
                     SPAN(w1, w1_of(s)), SPAN(w2, w2_of(s)), SPAN(offsets, s->E + 1), SPAN(dY, n * s->H)}));
  }
  cudaStream_t st = stream_of(stream);
  int sms = 0;
  TRY(train_setup(&sms));
  if (s->T == 0) return zero_weights(s, dw1, dw2, st);
  Carve c(ws);
  const FfnGradWs w = ffn_grad_ws(s, false, c);
  GatherArgs ga = {segments(s, offsets), false, nullptr, s->T, s->H, s->k, (int)ld_of(s->H), {xp, dY}, {w.xp, w.dyp}};
  CUDA_TRY(launch_train_gather(ga, sms, st), "row copy launch");
  FfnGrad f = {keep_bits, w.xp, w.dyp, w1, w2, offsets, z, z_scales, nullptr, nullptr, nullptr,
               w.hw, w.dz, dxp, dw1, dw2, w.dxp};
  return ffn_gradients(s, f, status, st);
}

size_t moet_router_probs_workspace_size(const moe_shape* s) {
  if (check_train_shape(s, false) != MOE_OK) return 0;
  Carve c(nullptr);
  probs_ws(s, c);
  return c.used + 1024;
}

int moet_router_probs(const moe_shape* s, const uint16_t* x, const uint16_t* w_router, const float* b_router,
                      float* probs, void* status, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_train_shape(s, false));
  CHECK_WS(moet_router_probs_workspace_size(s), "moet_router_probs_workspace_size");
  if (b_router && !aligned16(b_router)) return fail(MOE_ERR_INVALID_ARG, "b_router is not 16-byte aligned");
  if (s->T == 0) return MOE_OK;
  REQUIRE_PTR(x);
  REQUIRE_PTR(w_router);
  REQUIRE_PTR(probs);
  TRY(check_apart({SPAN(probs, (size_t)s->T * s->E), Span{status, MOE_WS_MIN_BYTES, "status"},
                   Span{ws, moet_router_probs_workspace_size(s), "ws"}},
                  {SPAN(x, (size_t)s->T * s->H), SPAN(w_router, (size_t)s->H * s->E), SPAN(b_router, s->E)}));
  int sms = 0;
  TRY(train_setup(&sms));
  Carve c(ws);
  return router_probs(s, sms, probs_ws(s, c), x, w_router, b_router, probs, status, stream_of(stream));
}

size_t moet_route_backward_workspace_size(const moe_shape* s) {
  if (check_train_shape(s, false) != MOE_OK) return 0;
  Carve c(nullptr);
  route_grad_ws(s, c);
  return c.used + 1024;
}

int moet_route_backward(const moe_shape* s, const uint16_t* x, const uint16_t* w_router, const int32_t* ids,
                        const float* weights, const float* probs, const float* dweights, uint16_t* dx,
                        uint16_t* dw_router, float* db, void* status, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_train_shape(s, false));
  CHECK_WS(moet_route_backward_workspace_size(s), "moet_route_backward_workspace_size");
  REQUIRE_PTR(dw_router);
  if (db && !aligned16(db)) return fail(MOE_ERR_INVALID_ARG, "db is not 16-byte aligned");
  if (s->T > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(w_router);
    REQUIRE_PTR(ids);
    REQUIRE_PTR(weights);
    if (s->gating == MOE_GATE_SOFTMAX_TOPK) REQUIRE_PTR(probs);
    REQUIRE_PTR(dweights);
    REQUIRE_PTR(dx);
    const size_t n = rows_of(s);
    TRY(check_apart({SPAN(dx, (size_t)s->T * s->H), SPAN(dw_router, (size_t)s->H * s->E), SPAN(db, s->E),
                     Span{status, MOE_WS_MIN_BYTES, "status"}, Span{ws, moet_route_backward_workspace_size(s), "ws"}},
                    {SPAN(x, (size_t)s->T * s->H), SPAN(w_router, (size_t)s->H * s->E), SPAN(ids, n), SPAN(weights, n),
                     SPAN(probs, s->gating == MOE_GATE_SOFTMAX_TOPK ? (size_t)s->T * s->E : 0), SPAN(dweights, n)}));
  }
  cudaStream_t st = stream_of(stream);
  int sms = 0;
  TRY(train_setup(&sms));
  if (s->T == 0) {
    TRY(zero(dw_router, (size_t)s->H * s->E * 2, st));
    return db ? zero(db, (size_t)s->E * 4, st) : MOE_OK;
  }
  Carve c(ws);
  const RouteGradWs r = route_grad_ws(s, c);
  GateBackwardArgs g = gate_args(s, r, w_router, ids, weights, probs);
  g.dw = dweights;
  RowsSumArgs sum = {};
  sum.T = s->T;
  sum.H = s->H;
  sum.k = s->k;
  sum.out = dx;
  return route_gradients(s, r, g, x, dw_router, db, nullptr, sum, status, st);
}

size_t moet_forward_workspace_size(const moe_shape* s) {
  if (check_train_shape(s, true) != MOE_OK) return 0;
  Carve c(nullptr);
  forward_ws(s, c);
  return c.used + 1024;
}

int moet_forward(const moe_shape* s, int32_t keep_bits, const uint16_t* x, const uint16_t* w_router,
                 const float* b_router, const uint16_t* w1, const uint16_t* w2, uint16_t* y, int32_t* ids,
                 float* weights, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* slot, void* z,
                 uint8_t* z_scales, int8_t* xk, uint8_t* xk_scales, float* probs, void* status, void* ws,
                 size_t ws_bytes, void* stream) {
  TRY(check_train_shape(s, true));
  TRY(check_bits(keep_bits));
  CHECK_WS(moet_forward_workspace_size(s), "moet_forward_workspace_size");
  REQUIRE_PTR(counts);
  REQUIRE_PTR(offsets);
  if (b_router && !aligned16(b_router)) return fail(MOE_ERR_INVALID_ARG, "b_router is not 16-byte aligned");
  if (s->T > 0) {
    REQUIRE_PTR(w1);
    REQUIRE_PTR(w2);
    REQUIRE_PTR(y);
    REQUIRE_PTR(z);
    if (keep_bits == 8) {
      REQUIRE_PTR(z_scales);
      REQUIRE_PTR(xk);
      REQUIRE_PTR(xk_scales);
    }
    if (s->gating == MOE_GATE_SOFTMAX_TOPK) REQUIRE_PTR(probs);
    REQUIRE_PTR(x);
    REQUIRE_PTR(w_router);
    REQUIRE_PTR(ids);
    REQUIRE_PTR(weights);
    REQUIRE_PTR(perm);
    REQUIRE_PTR(slot);
    const size_t n = rows_of(s), x8 = keep_bits == 8 ? s->T : 0;
    TRY(check_apart({SPAN(y, (size_t)s->T * s->H), SPAN(ids, n), SPAN(weights, n), SPAN(counts, s->E),
                     SPAN(offsets, s->E + 1), SPAN(perm, n), SPAN(slot, n), kept_span(s, keep_bits, z),
                     kept_scales_span(s, keep_bits, z_scales), SPAN(xk, x8 * s->H),
                     SPAN(xk_scales, x8 * (((size_t)s->H + 31) / 32)),
                     SPAN(probs, s->gating == MOE_GATE_SOFTMAX_TOPK ? (size_t)s->T * s->E : 0),
                     Span{status, MOE_WS_MIN_BYTES, "status"}, Span{ws, moet_forward_workspace_size(s), "ws"}},
                    {SPAN(x, (size_t)s->T * s->H), SPAN(w_router, (size_t)s->H * s->E), SPAN(b_router, s->E),
                     SPAN(w1, w1_of(s)), SPAN(w2, w2_of(s))}));
  }
  cudaStream_t st = stream_of(stream);
  int sms = 0;
  TRY(train_setup(&sms));
  Carve c(ws);
  const ForwardWs w = forward_ws(s, c);
  TRY(moe_route(s, x, w_router, b_router, ids, weights, counts, offsets, perm, slot, w.route, w.route_bytes,
                stream));
  if (s->T == 0) return MOE_OK;
  if (s->gating == MOE_GATE_SOFTMAX_TOPK)
    TRY(router_probs(s, sms, w.probs, x, w_router, b_router, probs, status, st));
  if (keep_bits == 8)
    CUDA_TRY(launch_quantize_a8(s->T, s->H, x, xk, xk_scales, sms, st), "quantize launch");
  GatherArgs ga = {segments(s, offsets), true, perm, s->T, s->H, s->k, (int)ld_of(s->H), {x, nullptr}, {w.xp, nullptr}};
  CUDA_TRY(launch_train_gather(ga, sms, st), "row copy launch");
  // the route's own status word is taken over by the next product
  TRY(fwd_product(s, keep_bits, w.xp, ld_of(s->H), w1, offsets, w.ffn.h, z, z_scales, static_cast<const int*>(w.route),
                  status, st));
  // the experts' outputs stay in fp32: y is rounded once
  TRY(plain_product(s, w.ffn.h, w2, offsets, nullptr, w.Y, status, st));
  RowsSumArgs ca = {};
  ca.rows32 = w.Y;
  ca.splits = row_split(rows_of(s), s->E, s->H, s->F).parts;
  ca.w = weights;
  ca.slot = slot;
  ca.T = s->T;
  ca.H = s->H;
  ca.k = s->k;
  ca.out = y;
  CUDA_TRY(launch_rows_sum(ca, st), "combine launch");
  return MOE_OK;
}

size_t moet_backward_workspace_size(const moe_shape* s, int32_t keep_bits) {
  if (check_train_shape(s, true) != MOE_OK || check_bits(keep_bits) != MOE_OK) return 0;
  Carve c(nullptr);
  backward_ws(s, keep_bits, c);
  return c.used + 1024;
}

int moet_backward(const moe_shape* s, int32_t keep_bits, const uint16_t* dy, const void* x,
                  const uint8_t* x_scales, const uint16_t* w_router, const uint16_t* w1, const uint16_t* w2,
                  const int32_t* ids, const float* weights, const int32_t* offsets, const int32_t* perm,
                  const int32_t* slot, const void* z, const uint8_t* z_scales, const float* probs,
                  uint16_t* dx, uint16_t* dw_router, float* db, uint16_t* dw1, uint16_t* dw2, void* status,
                  void* ws, size_t ws_bytes, void* stream) {
  TRY(check_train_shape(s, true));
  TRY(check_bits(keep_bits));
  CHECK_WS(moet_backward_workspace_size(s, keep_bits), "moet_backward_workspace_size");
  REQUIRE_PTR(dw_router);
  REQUIRE_PTR(dw1);
  REQUIRE_PTR(dw2);
  if (db && !aligned16(db)) return fail(MOE_ERR_INVALID_ARG, "db is not 16-byte aligned");
  if (s->T > 0) {
    REQUIRE_PTR(dy);
    REQUIRE_PTR(x);
    REQUIRE_PTR(w_router);
    REQUIRE_PTR(w1);
    REQUIRE_PTR(w2);
    REQUIRE_PTR(ids);
    REQUIRE_PTR(weights);
    REQUIRE_PTR(offsets);
    REQUIRE_PTR(perm);
    REQUIRE_PTR(slot);
    REQUIRE_PTR(z);
    if (keep_bits == 8) {
      REQUIRE_PTR(z_scales);
      REQUIRE_PTR(x_scales);
    }
    if (s->gating == MOE_GATE_SOFTMAX_TOPK) REQUIRE_PTR(probs);
    REQUIRE_PTR(dx);
    const size_t n = rows_of(s), th = (size_t)s->T * s->H;
    TRY(check_apart({SPAN(dx, th), SPAN(dw_router, (size_t)s->H * s->E), SPAN(db, s->E), SPAN(dw1, w1_of(s)),
                     SPAN(dw2, w2_of(s)), Span{status, MOE_WS_MIN_BYTES, "status"},
                     Span{ws, moet_backward_workspace_size(s, keep_bits), "ws"}},
                    {SPAN(dy, th), Span{x, th * (keep_bits / 8), "x"},
                     SPAN(x_scales, keep_bits == 8 ? (size_t)s->T * (((size_t)s->H + 31) / 32) : 0),
                     SPAN(w_router, (size_t)s->H * s->E), SPAN(w1, w1_of(s)), SPAN(w2, w2_of(s)), SPAN(ids, n),
                     SPAN(weights, n), SPAN(offsets, s->E + 1), SPAN(perm, n), SPAN(slot, n),
                     kept_span(s, keep_bits, z), kept_scales_span(s, keep_bits, z_scales),
                     SPAN(probs, s->gating == MOE_GATE_SOFTMAX_TOPK ? (size_t)s->T * s->E : 0)}));
  }
  cudaStream_t st = stream_of(stream);
  int sms = 0;
  TRY(train_setup(&sms));
  if (s->T == 0) {
    TRY(zero(dw_router, (size_t)s->H * s->E * 2, st));
    if (db) TRY(zero(db, (size_t)s->E * 4, st));
    return zero_weights(s, dw1, dw2, st);
  }
  Carve c(ws);
  const BackwardWs w = backward_ws(s, keep_bits, c);
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  if (keep_bits == 8) {
    CUDA_TRY(launch_dequantize_a8(s->T, s->H, static_cast<const int8_t*>(x), x_scales, w.x, sms, st),
             "dequantize launch");
    xb = w.x;
  }
  GatherArgs ga = {segments(s, offsets), false, perm, s->T, s->H, s->k, (int)ld_of(s->H), {xb, dy}, {w.ffn.xp, w.ffn.dyp}};
  CUDA_TRY(launch_train_gather(ga, sms, st), "row copy launch");
  FfnGrad f = {keep_bits, w.ffn.xp, w.ffn.dyp, w1, w2, offsets, z, z_scales, weights, perm, w.part,
               w.ffn.hw, w.ffn.dz, nullptr, dw1, dw2, w.ffn.dxp};
  TRY(ffn_gradients(s, f, status, st));
  GateBackwardArgs g = gate_args(s, w.route, w_router, ids, weights, probs);
  g.part = w.part;
  g.slot = slot;
  g.rows = (int)rows_of(s);
  g.units = (s->F + 63) / 64;
  RowsSumArgs sum = {};
  sum.rows32 = w.ffn.dxp;
  sum.splits = row_split(rows_of(s), s->E, s->H, s->F * halves(s)).parts;
  sum.slot = slot;
  sum.T = s->T;
  sum.H = s->H;
  sum.k = s->k;
  sum.out = dx;
  return route_gradients(s, w.route, g, xb, dw_router, db, w.dxr, sum, status, st);
}

}  // extern "C"
