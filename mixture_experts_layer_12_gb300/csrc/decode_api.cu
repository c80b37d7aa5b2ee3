// decode_api.cu -- the C ABI declared in include/moe_decode.h: argument
// checks, workspace layout, tensor maps and the two launches of a call on the
// caller's stream.  No allocation and no host synchronisation.
#include <mutex>

#include "api_internal.h"
#include "decode_internal.h"

using namespace moe;

namespace {

cudaError_t decode_set_attributes() {
  cudaError_t e = decode_route_set_attributes();
  if (e == cudaSuccess) e = decode_ffn_bf16_set_attributes();
  if (e == cudaSuccess) e = decode_ffn_pair_set_attributes();
  if (e == cudaSuccess) e = decode_ffn_q4_32_set_attributes();
  if (e == cudaSuccess) e = decode_ffn_q4_64_set_attributes();
  if (e == cudaSuccess) e = decode_ffn_q4_128_set_attributes();
  return e;
}

std::mutex g_mu;
bool g_ready[kMaxDevices];

// device_setup() and, on a device's first use here, the attributes of these
// kernels: their code is loaded by this, 1.6 ms and 2 MB of device memory that
// callers of the other entry points do not need.
int decode_setup(int* sms) {
  int rc = device_setup(sms);
  if (rc != MOE_OK) return rc;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_ready[dev]) {
    if ((e = decode_set_attributes()) != cudaSuccess) return cuda_fail(e, "decode attributes");
    g_ready[dev] = true;
  }
  return MOE_OK;
}

cudaError_t launch_decode_ffn(const DecFfnMaps& m, const DecFfnArgs& a, int ctas, cudaStream_t st) {
  switch (a.group) {
    case 0: return launch_decode_ffn_bf16(m, a, ctas, st);
    case kDecPair: return launch_decode_ffn_pair(m, a, ctas, st);
    case 32: return launch_decode_ffn_q4_32(m, a, ctas, st);
    case 64: return launch_decode_ffn_q4_64(m, a, ctas, st);
    default: return launch_decode_ffn_q4_128(m, a, ctas, st);
  }
}

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Workspace: [control block | entries | partial tiles of both products | expert
// outputs of whole items, fp32 | h].  The control block is cleared by the first
// kernel of every call.
struct Layout {
  size_t entries, parts, parts2, yfull, h, total;
  int max_entries, row_cap;
};

// Rows of an entry at most.  The kernel is built for 8, 16, 32 and 64 rows; an
// expert or segment with more is cut into several entries, which read its
// weights once each.  With 4-bit weights the cost of an entry grows with the
// rows it has room for (registers, ring space, products): room for the average
// and 1.4 times its square root more, what an even choice of experts hardly
// exceeds (37 rows over 64 segments: 27 us with entries of up to 64 rows, 18
// with 8; 32 rows over 8 experts: 108 us with 16, 100 with 8).  With bf16
// weights reading them twice costs more than room does: 3 square roots.
// Uneven choices pay for that: 64 tokens that all choose the same 2 of 8 experts of
// 4096 x 14336 read their weights twice (bf16 137 us, 4 bits 134; one reading takes 69
// and 18), 64 that choose the same one of 128 of 2048 x 1408 eight times (37 and 27 us).
// `most`: rows that one can hold.
int row_block_of(bool q4, int rows, int parts, int most) {
  const int avg = (rows + parts - 1) / parts;
  int root = 0;
  while ((root + 1) * (root + 1) <= (q4 ? 2 : 9) * avg) ++root;
  int rb = 8;
  while (rb < kDecRows && rb < avg + root && rb < most) rb *= 2;
  return rb;
}

// pair: the first product's partial tiles are a gate's and an up projection's
Layout layout_of(int rows, int row_cap, int max_entries, int H, int F, bool layer, bool pair) {
  Layout L;
  L.max_entries = max_entries;
  L.row_cap = row_cap;
  L.entries = kDecEntryOffset;
  L.parts = L.entries + up((size_t)max_entries * sizeof(DecEntry), 1024);
  const size_t tiles = (size_t)kDecMaxCtas * 2 * row_cap * kDecBN * 4;
  L.parts2 = L.parts + tiles * (pair ? 2 : 1);
  L.yfull = L.parts2 + (layer ? tiles : 0);
  L.h = L.yfull + (layer ? up((size_t)rows * H * 4, 1024) : 0);
  L.total = L.h + (layer ? up((size_t)rows * F * 2, 1024) : 0);
  return L;
}

// ceil(n_e / block) summed over at most `parts` experts or segments with n_e
// rows, `rows` in all
int max_entries_of(int rows, int parts, int block) {
  return rows < parts ? rows : parts + (rows - parts) / block;
}

// How the first product of gated bf16 experts is cut (kDecPair).
// Chunks of 64 gate and 64 up columns are rows of 128 bytes, which memory delivers
// a quarter more slowly than the 256 of 128 columns (64 experts of 2048 x 1408, 32
// tokens: 204 us, with alternating chunks of 128 columns 157); but those are dealt
// out in pairs, 32 KB, and where a CTA has few of them one more or less is what
// counts (one token, 9 pairs per CTA: 24.8 us, 25.3 with pairs; 2 tokens, 18 pairs:
// 35.8, 34.5).  With 4 bits 64 columns are 256 bytes.
bool pair_of(const moe_shape* s, bool q4) {
  if (q4 || s->expert_act != MOE_EXPERT_SWIGLU) return false;
  const int64_t hit = (int64_t)s->T * s->k < s->E ? s->T * s->k : s->E;
  const int64_t nb = (s->F + kDecBN - 1) / kDecBN, kc = (s->H + kDecKC16 - 1) / kDecKC16;
  return hit * nb * kc >= 12 * kDecMaxCtas;
}

Layout layer_layout(const moe_shape* s, bool q4) {
  const int rows = s->T > 0 ? s->T * s->k : 1;
  const int block = row_block_of(q4, rows, s->E, s->T);
  return layout_of(rows, block, max_entries_of(rows, s->E, block), s->H, s->F, true,
                   pair_of(s, q4));
}

Layout matvec_layout(int rows, int n_segments) {
  const int r = rows > 0 ? rows : 1;
  const int block = row_block_of(true, r, n_segments, r);
  return layout_of(r, block, max_entries_of(r, n_segments, block), 0, 0, false, false);
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

int check_layer(const moe_shape* s) {
  int rc = check_shape(s, true);
  if (rc != MOE_OK) return rc;
  if (s->T > MOED_MAX_TOKENS)
    return fail(MOE_ERR_UNSUPPORTED, "T = %d: the decode operators take at most %d tokens", s->T,
                MOED_MAX_TOKENS);
  if ((int64_t)s->F * 2 > (int64_t)1 << 30 || (int64_t)s->H > (int64_t)1 << 30)
    return fail(MOE_ERR_UNSUPPORTED, "H = %d, F = %d: too large", s->H, s->F);
  return MOE_OK;
}

int check_group(int32_t group) {
  if (group != 32 && group != 64 && group != 128)
    return fail(MOE_ERR_UNSUPPORTED, "group = %d: need 32, 64 or 128", group);
  return MOE_OK;
}

int check_q4_layer(const moe_shape* s, int32_t group) {
  int rc = check_group(group);
  if (rc != MOE_OK) return rc;
  if (s->H % group != 0 || s->F % group != 0)
    return fail(MOE_ERR_UNSUPPORTED, "H = %d, F = %d: need multiples of the group (%d)", s->H, s->F, group);
  return MOE_OK;
}

int check_q4(int32_t E, int32_t K, int32_t N, int32_t group) {
  int rc = check_group(group);
  if (rc != MOE_OK) return rc;
  if (E < 1 || E > kMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "E = %d: need 1 <= E <= %d", E, kMaxExperts);
  if (K < group || K % group != 0 || K > 1 << 24)
    return fail(MOE_ERR_UNSUPPORTED, "K = %d: need a multiple of the group (%d), at most 2^24", K, group);
  if (N < 8 || N % 8 != 0 || N > 1 << 24)
    return fail(MOE_ERR_UNSUPPORTED, "N = %d: need N >= 8, N %% 8 == 0, at most 2^24", N);
  // one thread per 64 weights, one block per 256 of them, on a 31-bit grid
  if ((int64_t)E * (K / 8) * (N / 8) > (int64_t)1 << 38)
    return fail(MOE_ERR_UNSUPPORTED, "E * K * N = %d * %d * %d: too large", E, K, N);
  return MOE_OK;
}

// The weights' tensor map (see DecFfnMaps): W [E, K, N] bf16, or words
// [E, K/8, N]; `half`: columns of a gate / up half (N where there is none).
int map_weights(CUtensorMap* m, int* blocked, const void* w, bool q4, int E, int K, int N, int half, bool pair,
                const char* what) {
  const uint64_t rows = q4 ? K / 8 : K;
  const uint64_t esize = q4 ? 4 : 2;
  const uint64_t blk = 128 / esize;
  const uint32_t box_rows = q4 ? kDecKC4 / 8 : kDecKC16;
  const CUtensorMapDataType type = q4 ? CU_TENSOR_MAP_DATA_TYPE_INT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const bool gated = half != N;
  *blocked = half % (int)blk == 0;
  if (*blocked) {
    const uint64_t dims[4] = {blk, rows, (uint64_t)N / blk, (uint64_t)E};
    const uint64_t strides[3] = {(uint64_t)N * esize, 128, rows * N * esize};
    const uint32_t box[4] = {(uint32_t)blk, box_rows, (uint32_t)((gated && !pair ? 64 : kDecBN) / blk), 1};
    return encode_map_as(m, type, CU_TENSOR_MAP_SWIZZLE_128B, w, 4, dims, strides, box, what);
  }
  const uint64_t dims[3] = {(uint64_t)N, rows, (uint64_t)E};
  const uint64_t strides[2] = {(uint64_t)N * esize, rows * N * esize};
  const uint32_t box[3] = {(uint32_t)blk, box_rows, 1};
  return encode_map_as(m, type, CU_TENSOR_MAP_SWIZZLE_128B, w, 3, dims, strides, box, what);
}

int empty_call(void* ws, int32_t* counts, int32_t* offsets, int E, cudaStream_t st) {
  cudaError_t e = launch_clear_status(static_cast<int*>(ws), st, true);
  if (e == cudaSuccess && counts) e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)E, st);
  if (e == cudaSuccess && offsets) e = cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (size_t)(E + 1), st);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "clearing an empty call's outputs");
}

// Chunks worth a CTA of their own where a product is too small for all CTAs: a
// chunk is read in ~0.37 us and a partial tile added in ~0.25, so n chunks per
// CTA and K-chunks / n tiles per item cost least at n = sqrt(0.7 K-chunks).
int least_chunks(int kc) {
  int n = 1;
  while (10 * (n + 1) * (n + 1) <= 7 * kc && n < 64) ++n;
  return n;
}

// The streaming kernel counts a product's chunks, times its CTAs, in 32 bits.
int check_chunks(int64_t entries, int64_t nb, int64_t kc) {
  if (nb * kc > ((int64_t)1 << 32) / kDecMaxCtas || entries * nb * kc >= ((int64_t)1 << 32) / kDecMaxCtas)
    return fail(MOE_ERR_UNSUPPORTED, "%lld x %lld x %lld weight tiles: too many", (long long)entries,
                (long long)nb, (long long)kc);
  return MOE_OK;
}

struct Weights {
  bool q4;
  int group;
  const void *w1, *s1, *w2, *s2;
};

// missing: CTAs that the grid barriers wait for in vain (the self-test)
int forward(const moe_shape* s, const Weights& wt, const uint16_t* x, const uint16_t* w_router,
            const float* b_router, uint16_t* y, int32_t* ids, float* weights, int32_t* counts,
            int32_t* offsets, int32_t* perm, int32_t* slot, void* ws, size_t ws_bytes,
            void* stream, uint64_t wait_limit_ns = kWaitLimitNs, int missing = 0) {
  int rc;
  REQUIRE_PTR(ws);
  const Layout L = layer_layout(s, wt.q4);
  if (ws_bytes < L.total)
    return fail(MOE_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed (moed_workspace_size)",
                ws_bytes, L.total);
  REQUIRE_PTR(counts);
  REQUIRE_PTR(offsets);
  if (b_router && !aligned16(b_router)) return fail(MOE_ERR_INVALID_ARG, "b_router is not 16-byte aligned");
  if (s->T > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(w_router);
    REQUIRE_PTR(wt.w1);
    REQUIRE_PTR(wt.w2);
    if (wt.q4) {
      REQUIRE_PTR(wt.s1);
      REQUIRE_PTR(wt.s2);
    }
    REQUIRE_PTR(y);
    REQUIRE_PTR(ids);
    REQUIRE_PTR(weights);
    REQUIRE_PTR(perm);
    REQUIRE_PTR(slot);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  if ((rc = decode_setup(&sms)) != MOE_OK) return rc;
  if (s->T == 0) return empty_call(ws, counts, offsets, s->E, st);

  const bool swiglu = s->expert_act == MOE_EXPERT_SWIGLU;
  const int N1 = swiglu ? 2 * s->F : s->F;
  DecFfnMaps maps;
  int blocked1 = 0, blocked2 = 0;
  const bool pair = pair_of(s, wt.q4);
  if ((rc = map_weights(&maps.w1, &blocked1, wt.w1, wt.q4, s->E, s->H, N1, s->F, pair, "W1")) != MOE_OK) return rc;
  if ((rc = map_weights(&maps.w2, &blocked2, wt.w2, wt.q4, s->E, s->F, s->H, s->H, false, "W2")) != MOE_OK) return rc;

  const int kc = wt.q4 ? kDecKC4 : kDecKC16;
  const int cols1 = swiglu && !pair ? 64 : kDecBN;  // columns of h per item
  const int nb1 = (s->F + cols1 - 1) / cols1, kc1 = (s->H + kc - 1) / kc;
  const int nb2 = (s->H + kDecBN - 1) / kDecBN, kc2 = (s->F + kc - 1) / kc;
  if ((rc = check_chunks(L.max_entries, nb1, kc1)) != MOE_OK) return rc;
  if ((rc = check_chunks(L.max_entries, nb2, kc2)) != MOE_OK) return rc;

  DecRouteArgs ra;
  ra.x = x;
  ra.w = w_router;
  ra.bias = b_router;
  ra.T = s->T;
  ra.H = s->H;
  ra.E = s->E;
  ra.k = s->k;
  ra.capacity = (int)capacity_of(s);
  ra.gating = s->gating;
  ra.ids = ids;
  ra.weights = weights;
  ra.counts = counts;
  ra.offsets = offsets;
  ra.perm = perm;
  ra.slot = slot;
  ra.ctrl = static_cast<int*>(ws);
  ra.entries = at<DecEntry>(ws, L.entries);
  ra.row_block = L.row_cap;
  cudaError_t e = launch_decode_route(ra, st);
  if (e != cudaSuccess) return cuda_fail(e, "decode route launch");

  DecFfnArgs fa = {};
  fa.ctrl = static_cast<const int*>(ws);
  fa.entries = ra.entries;
  fa.max_entries = L.max_entries;
  fa.barrier = at<unsigned>(ws, kDecBarrierOffset);
  fa.item_counts = at<unsigned>(ws, kDecItemOffset);
  fa.parts = at<float>(ws, L.parts);
  fa.row_cap = L.row_cap;
  fa.parts2 = at<float>(ws, L.parts2);
  fa.yfull = at<float>(ws, L.yfull);
  fa.h = at<uint16_t>(ws, L.h);
  fa.s1 = static_cast<const uint16_t*>(wt.s1);
  fa.s2 = static_cast<const uint16_t*>(wt.s2);
  fa.blocked1 = blocked1;
  fa.blocked2 = blocked2;
  fa.x = x;
  fa.perm = perm;
  fa.slot = slot;
  fa.gate = weights;
  fa.y = y;
  fa.T = s->T;
  fa.k = s->k;
  fa.act = swiglu ? kDecSwiGLU : kDecGelu;
  fa.group = pair ? kDecPair : wt.group;
  fa.K1 = s->H;
  fa.N1 = s->F;
  fa.nb1 = nb1;
  fa.kc1 = kc1;
  fa.least1 = least_chunks(pair ? kc1 / 2 : kc1);  // (a pair takes twice the time)
  fa.least2 = least_chunks(kc2);
  fa.K2 = s->F;
  fa.N2 = s->H;
  fa.nb2 = nb2;
  fa.kc2 = kc2;
  fa.status = static_cast<int*>(ws);
  fa.wait_limit_ns = wait_limit_ns;
  const int ctas = sms < kDecMaxCtas ? sms : kDecMaxCtas;
  fa.arrivals = (uint32_t)(ctas + missing);
  e = launch_decode_ffn(maps, fa, ctas, st);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "decode expert launch");
}

}  // namespace

extern "C" {

size_t moed_workspace_size(const moe_shape* s) {
  if (check_layer(s) != MOE_OK) return 0;
  const size_t a = layer_layout(s, false).total, b = layer_layout(s, true).total;
  return a > b ? a : b;
}

int moed_forward(const moe_shape* s, const uint16_t* x, const uint16_t* w_router,
                 const float* b_router, const uint16_t* w1, const uint16_t* w2, uint16_t* y,
                 int32_t* ids, float* weights, int32_t* counts, int32_t* offsets, int32_t* perm,
                 int32_t* slot, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_layer(s);
  if (rc != MOE_OK) return rc;
  const Weights wt{false, 0, w1, nullptr, w2, nullptr};
  return forward(s, wt, x, w_router, b_router, y, ids, weights, counts, offsets, perm, slot, ws,
                 ws_bytes, stream);
}

int moed_forward_q4(const moe_shape* s, int32_t group, const uint16_t* x, const uint16_t* w_router,
                    const float* b_router, const uint32_t* w1_codes, const uint16_t* w1_scales,
                    const uint32_t* w2_codes, const uint16_t* w2_scales, uint16_t* y, int32_t* ids,
                    float* weights, int32_t* counts, int32_t* offsets, int32_t* perm,
                    int32_t* slot, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_layer(s);
  if (rc != MOE_OK) return rc;
  if ((rc = check_q4_layer(s, group)) != MOE_OK) return rc;
  const Weights wt{true, group, w1_codes, w1_scales, w2_codes, w2_scales};
  return forward(s, wt, x, w_router, b_router, y, ids, weights, counts, offsets, perm, slot, ws,
                 ws_bytes, stream);
}

int moed_selftest_wait_timeout(const moe_shape* s, int32_t group, const uint16_t* x,
                               const uint16_t* w_router, const float* b_router, const void* w1,
                               const uint16_t* w1_scales, const void* w2, const uint16_t* w2_scales,
                               uint16_t* y, int32_t* ids, float* weights, int32_t* counts,
                               int32_t* offsets, int32_t* perm, int32_t* slot, void* ws,
                               size_t ws_bytes, uint64_t limit_ns, void* stream) {
  int rc = check_layer(s);
  if (rc != MOE_OK) return rc;
  if (group != 0 && (rc = check_q4_layer(s, group)) != MOE_OK) return rc;
  if (limit_ns < 1000 || limit_ns > kWaitLimitNs)
    return fail(MOE_ERR_INVALID_ARG, "limit_ns = %llu: need 1e3 .. 1e9", (unsigned long long)limit_ns);
  const Weights wt{group != 0, group, w1, w1_scales, w2, w2_scales};
  return forward(s, wt, x, w_router, b_router, y, ids, weights, counts, offsets, perm, slot, ws,
                 ws_bytes, stream, limit_ns, 1);
}

size_t moed_matvec_q4_workspace_size(int32_t rows, int32_t n_segments, int32_t K, int32_t N) {
  if (rows < 0 || rows > MOED_MAX_ROWS || n_segments < 1 || n_segments > kMaxExperts || K < 32 || N < 8) {
    fail(MOE_ERR_UNSUPPORTED, "rows = %d (0..%d), n_segments = %d (1..%d), K = %d, N = %d", rows,
         MOED_MAX_ROWS, n_segments, kMaxExperts, K, N);
    return 0;
  }
  return matvec_layout(rows, n_segments).total;
}

int moed_matvec_q4(int32_t rows, int32_t K, int32_t N, int32_t E, int32_t group, int32_t n_segments,
                   const uint16_t* x, const uint32_t* codes, const uint16_t* scales,
                   const int32_t* seg_offsets, uint16_t* y, void* ws, size_t ws_bytes,
                   void* stream) {
  int rc = check_q4(E, K, N, group);
  if (rc != MOE_OK) return rc;
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %d < 0", rows);
  if (rows > MOED_MAX_ROWS)
    return fail(MOE_ERR_UNSUPPORTED, "rows = %d: at most %d", rows, MOED_MAX_ROWS);
  if (n_segments < 1 || n_segments > kMaxExperts)
    return fail(MOE_ERR_INVALID_ARG, "n_segments = %d, must be 1..%d", n_segments, kMaxExperts);
  REQUIRE_PTR(ws);
  const Layout L = matvec_layout(rows, n_segments);
  if (ws_bytes < L.total)
    return fail(MOE_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed (moed_matvec_q4_workspace_size)",
                ws_bytes, L.total);
  if (rows > 0) {
    REQUIRE_PTR(x);
    REQUIRE_PTR(codes);
    REQUIRE_PTR(scales);
    if (seg_offsets || n_segments != 1) REQUIRE_PTR(seg_offsets);  // null: one segment, all rows
    REQUIRE_PTR(y);
    // rows of y are finished while others of x are still being read
    if (x < y + (size_t)rows * N && y < x + (size_t)rows * K)
      return fail(MOE_ERR_INVALID_ARG, "y overlaps x");
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int sms = 0;
  if ((rc = decode_setup(&sms)) != MOE_OK) return rc;
  if (rows == 0) return empty_call(ws, nullptr, nullptr, 0, st);

  const int nb = (N + kDecBN - 1) / kDecBN, kc = (K + kDecKC4 - 1) / kDecKC4;
  if ((rc = check_chunks(L.max_entries, nb, kc)) != MOE_OK) return rc;
  DecFfnMaps maps;
  int blocked = 0;
  if ((rc = map_weights(&maps.w1, &blocked, codes, true, E, K, N, N, false, "W")) != MOE_OK) return rc;
  maps.w2 = maps.w1;  // not used

  DecPrepArgs pa;
  pa.seg_offsets = seg_offsets;
  pa.n_segments = n_segments;
  pa.rows = rows;
  pa.E = E;
  pa.ctrl = static_cast<int*>(ws);
  pa.entries = at<DecEntry>(ws, L.entries);
  pa.max_entries = L.max_entries;
  pa.row_block = L.row_cap;
  cudaError_t e = launch_decode_prep(pa, st);
  if (e != cudaSuccess) return cuda_fail(e, "entry list launch");

  DecFfnArgs fa = {};
  fa.ctrl = static_cast<const int*>(ws);
  fa.entries = pa.entries;
  fa.max_entries = L.max_entries;
  fa.barrier = at<unsigned>(ws, kDecBarrierOffset);
  fa.item_counts = at<unsigned>(ws, kDecItemOffset);
  fa.parts = at<float>(ws, L.parts);
  fa.row_cap = L.row_cap;
  fa.s1 = scales;
  fa.blocked1 = blocked;
  fa.x = x;
  fa.y = y;
  fa.T = rows;
  fa.k = 1;
  fa.act = kDecNone;
  fa.group = group;
  fa.K1 = K;
  fa.N1 = N;
  fa.nb1 = nb;
  fa.kc1 = kc;
  fa.least1 = least_chunks(kc);
  fa.least2 = 1;
  fa.status = static_cast<int*>(ws);
  fa.wait_limit_ns = kWaitLimitNs;
  const int ctas = sms < kDecMaxCtas ? sms : kDecMaxCtas;
  fa.arrivals = (uint32_t)ctas;
  e = launch_decode_ffn(maps, fa, ctas, st);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "matrix-vector launch");
}

int moed_quantize_q4(int32_t E, int32_t K, int32_t N, int32_t group, const uint16_t* w,
                     uint32_t* codes, uint16_t* scales, void* stream) {
  int rc = check_q4(E, K, N, group);
  if (rc != MOE_OK) return rc;
  REQUIRE_PTR(w);
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  int sms = 0;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  cudaError_t e = launch_quantize_q4(E, K, N, group, w, codes, scales, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "quantize launch");
}

int moed_dequantize_q4(int32_t E, int32_t K, int32_t N, int32_t group, const uint32_t* codes,
                       const uint16_t* scales, uint16_t* w, void* stream) {
  int rc = check_q4(E, K, N, group);
  if (rc != MOE_OK) return rc;
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  REQUIRE_PTR(w);
  int sms = 0;
  if ((rc = device_setup(&sms)) != MOE_OK) return rc;
  cudaError_t e = launch_dequantize_q4(E, K, N, group, codes, scales, w, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "dequantize launch");
}

}  // extern "C"
