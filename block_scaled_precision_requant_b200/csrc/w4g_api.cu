// C ABI of the integer 4-bit projections, the expert router and combine, and
// the expert MLP: argument checks and launches.  Declarations and the
// contract of every entry point are in include/bsr.h.
#include <mutex>

#include <cuda_runtime.h>

#include "bsr.h"
#include "kernels.h"
#include "w4g.h"

namespace bsr {
bsr_status library_status_word(int** out);
bsr_status report(bsr_status st, const char* fmt, ...);
}  // namespace bsr

namespace {

using bsr::report;

bsr_status ok() { return report(BSR_OK, "%s", ""); }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bsr_status cuda_status(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return report(BSR_ECUDA, "%s: %s", what, cudaGetErrorString(e));
  return ok();
}

struct Device {
  int num_sms = 0;
  size_t smem_optin = 0;
  int* status = nullptr;
};
Device g_device[64];
std::mutex g_device_mu;

// The current device's facts (an sm_100 device, else BSR_ENODEV).
bsr_status device(Device& out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return report(BSR_ENODEV, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= 64) return report(BSR_ENODEV, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_device_mu);
  Device& d = g_device[dev];
  if (d.num_sms == 0) {
    int* status = nullptr;
    const bsr_status st = bsr::library_status_word(&status);
    if (st != BSR_OK) return st;
    int sms = 0, smem = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess)
      return report(BSR_ENODEV, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    d.smem_optin = (size_t)smem;
    d.status = status;
    d.num_sms = sms;
  }
  out = d;
  return BSR_OK;
}

// The kernels count rows and elements of K in 32 bits, up to a tile past the end.
bool dim_ok(int64_t x) { return x >= 0 && x <= BSR_W4G_MAX_DIM; }

// Everything about a 4-bit weight that does not depend on its pointers.
bsr_status check_format(const bsr_w4g_weight* w, const char* who, int64_t k) {
  if (!w) return report(BSR_EINVAL, "%s: null weight", who);
  if (w->scale_type != BSR_W4G_SCALE_BF16 && w->scale_type != BSR_W4G_SCALE_FP16)
    return report(BSR_EINVAL, "%s: unknown scale type %d", who, w->scale_type);
  if (w->group != 32 && w->group != 64 && w->group != 128)
    return report(BSR_ESHAPE, "%s: group %d is not 32, 64 or 128", who, w->group);
  if (k <= 0 || k % w->group != 0)
    return report(BSR_ESHAPE, "%s: K=%lld must be a positive multiple of the group %d", who, (long long)k, w->group);
  return BSR_OK;
}

bsr_status check_weight(const bsr_w4g_weight* w, const char* who) {
  if (!w->q || !w->scale) return report(BSR_EINVAL, "%s: null weight pointer", who);
  if (!aligned(w->q, 16) || !aligned(w->scale, 2))
    return report(BSR_EALIGN, "%s: codes must be 16-byte aligned, scales 2-byte aligned", who);
  return BSR_OK;
}

bsr::W4gArgs make_args(const uint16_t* a, int64_t a_rows, const int32_t* offsets, const int32_t* rows,
                       const bsr_w4g_weight* w, uint16_t* out, int64_t r, int64_t experts, int64_t n, int64_t k) {
  bsr::W4gArgs g = {};
  g.a = a;
  g.offsets = offsets;
  g.rows = rows;
  g.q = w->q;
  g.scale = w->scale;
  g.zero = w->zero;
  g.out = out;
  g.a_rows = a_rows;
  g.rows_max = r;
  g.experts = (int)experts;
  g.n = (int)n;
  g.k = (int)k;
  g.group = w->group;
  g.half_scale = w->scale_type == BSR_W4G_SCALE_FP16 ? 1 : 0;
  return g;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point, so the
// library does not link libcuda directly.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bsr_status encode_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                     uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw,
                     const char* what) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return report(BSR_ECUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {pitch_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return report(BSR_ECUDA, "cuTensorMapEncodeTiled(%s) failed: %d", what, (int)r);
  return BSR_OK;
}

// At most this many rows never take the tensor-core kernel.
bool few_rows(int64_t r, int64_t experts) { return r <= bsr::kW4gFewRows * experts; }

// One product, every check and tensor map made before its launch.  `gather`:
// it takes its rows in order, from the buffer that the plan was given.
struct Product {
  bsr::W4gArgs g;
  bsr::W4gPlan plan;
  bool gather = false;
  CUtensorMap q, a;
};

bsr_status plan_product(Product& p, const bsr::W4gArgs& g, uint16_t* ordered, const Device& d) {
  p.g = g;
  p.plan = bsr::w4g_plan(g, d.num_sms);
  const uint64_t wrows = (uint64_t)g.experts * (uint64_t)g.n, wpitch = (uint64_t)g.k / 2;
  if (p.plan.few) {
    return encode_2d(&p.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.q, wpitch, wrows, wpitch, 128, bsr::kW4gGemvRows,
                     CU_TENSOR_MAP_SWIZZLE_128B, "w4g codes");
  }
  const bsr_status st = encode_2d(&p.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.q, wpitch, wrows, wpitch, 64, 128,
                                  CU_TENSOR_MAP_SWIZZLE_64B, "w4g codes");
  if (st != BSR_OK) return st;
  if (g.rows) {  // the tensor-core kernel takes its rows in order: they are gathered first
    p.gather = true;
    p.g.a = ordered;
    p.g.a_rows = g.rows_max;
    p.g.rows = nullptr;
  }
  return encode_2d(&p.a, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.g.a, (uint64_t)g.k, (uint64_t)p.g.a_rows,
                   (uint64_t)g.k * 2, 64, (uint32_t)p.plan.gemm.bm, CU_TENSOR_MAP_SWIZZLE_128B, "w4g activations");
}

bsr_status run_product(const Product& p, const Device& d, void* stream) {
  return cuda_status(p.plan.few ? bsr::launch_w4g_gemv(p.q, p.g, p.plan.gemv, d.status, as_stream(stream))
                                : bsr::launch_w4g_gemm(p.q, p.a, p.g, p.plan.gemm, d.status, as_stream(stream)),
                     "w4g projection launch");
}

bsr_status check_route_dims(const char* who, int64_t tokens, int64_t experts, int64_t top_k) {
  if (tokens < 0 || experts < 1 || experts > bsr::kRouteMaxExperts || top_k < 1 || top_k > experts ||
      top_k > bsr::kRouteMaxTopK || tokens > BSR_W4G_MAX_DIM / top_k)
    return report(BSR_EINVAL, "%s: tokens=%lld experts=%lld top_k=%lld (1 <= experts <= %d, 1 <= top_k <= "
                              "min(experts, %d), tokens * top_k <= 2^31 - 256)",
                  who, (long long)tokens, (long long)experts, (long long)top_k, bsr::kRouteMaxExperts,
                  bsr::kRouteMaxTopK);
  return BSR_OK;
}

bsr_status check_logits(const char* who, const void* logits, int logits_type, unsigned flags) {
  if (logits_type != BSR_MOE_LOGITS_F32 && logits_type != BSR_MOE_LOGITS_BF16)
    return report(BSR_EINVAL, "%s: unknown logits type %d", who, logits_type);
  if (flags & ~(unsigned)BSR_MOE_RENORMALIZE) return report(BSR_EINVAL, "%s: unknown flags 0x%x", who, flags);
  if (!logits) return report(BSR_EINVAL, "%s: null logits", who);
  if (!aligned(logits, logits_type == BSR_MOE_LOGITS_BF16 ? 2 : 4))
    return report(BSR_EALIGN, "%s: logits must be aligned to their type", who);
  return BSR_OK;
}

// Scratch of the expert MLP: the route's results and scratch, the gathered rows,
// then the gate, up, hidden (their SiLU product) and down rows.
struct MlpLayout {
  size_t ids, weights, offsets, rows, pos, route, ordered, gate, up, hidden, down, total;
};
// Its size stays below 2^62 bytes (and a little): the rows alone are 2 (3 inner +
// 2 k) bytes per pair.
bool mlp_fits(int64_t tokens, int64_t top_k, int64_t inner, int64_t k) {
  return tokens * top_k <= (int64_t(1) << 61) / (3 * inner + 2 * k);
}
MlpLayout mlp_layout(int64_t tokens, int64_t experts, int64_t top_k, int64_t inner, int64_t k) {
  const size_t pairs = (size_t)tokens * (size_t)top_k;
  MlpLayout L;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  L.ids = take(pairs * 4);
  L.weights = take(pairs * 4);
  L.offsets = take(((size_t)experts + 1) * 4);
  L.rows = take(pairs * 4);
  L.pos = take(pairs * 4);
  L.route = take(bsr::route_scratch_bytes(tokens, (int)experts));
  L.ordered = take(few_rows((int64_t)pairs, experts) ? 0 : pairs * (size_t)k * 2);
  L.gate = take(pairs * (size_t)inner * 2);
  L.up = take(pairs * (size_t)inner * 2);
  L.hidden = take(pairs * (size_t)inner * 2);
  L.down = take(pairs * (size_t)k * 2);
  L.total = at;
  return L;
}

}  // namespace

namespace bsr {

// The decode kernel reads the weight at more than the tensor-core kernel's
// rate and splits K, but its work grows with every 8 rows of an expert; the
// tensor-core kernel's time is that of whole tiles.  Each plan estimates its
// own, and past 16 rows per expert (two tiles of the decode kernel's widest
// item) or 4096 in all its is never the shorter.  (Measured, us, decode /
// tensor-core: 14336 x 4096 at 8 rows 14.0 / 17.5, at 12 21.0 / 17.6, with
// groups of 32 24.7 / 27.7; 4096 x 4096 at 8 rows 8.3 / 9.2, at 12 9.9 / 9.2; 128
// experts of 1536 x 2048 at 5 rows each 64 / 87, at 8 99 / 87, with groups of 32
// 117 / 151; 8 experts of 14336 x 4096 at 6 rows each 75 / 104, at 8 116 / 103.
// The estimates miss by up to 15% beside the crossover: 2048 x 2048 at 8 rows
// takes the tensor cores, 5.2 / 6.0, the 128 experts with groups of 32 at 12 rows
// each too, 132 / 150.)
W4gPlan w4g_plan(const W4gArgs& g, int num_sms) {
  W4gPlan p;
  p.gemm = w4g_gemm_plan(g, num_sms);
  p.few = few_rows(g.rows_max, g.experts);
  if (p.few || (g.rows_max <= 16LL * g.experts && g.rows_max <= 4096)) {
    p.gemv = w4g_gemv_plan(g, num_sms);
    p.few = p.few || p.gemv.us < p.gemm.us;
  }
  return p;
}

}  // namespace bsr

extern "C" {

bsr_status bsr_w4g_proj(const uint16_t* a, const bsr_w4g_weight* w, uint16_t* out, int64_t m, int64_t n, int64_t k,
                        void* stream) {
  bsr_status st = check_format(w, "bsr_w4g_proj", k);
  if (st != BSR_OK) return st;
  if (!dim_ok(m) || !dim_ok(n) || !dim_ok(k))
    return report(BSR_EINVAL, "dimension out of range (m=%lld n=%lld k=%lld)", (long long)m, (long long)n,
                  (long long)k);
  if (m == 0 || n == 0) return ok();
  if (!a || !out) return report(BSR_EINVAL, "bsr_w4g_proj: null pointer");
  if ((st = check_weight(w, "bsr_w4g_proj")) != BSR_OK) return st;
  if (!aligned(a, 16) || !aligned(out, 2))
    return report(BSR_EALIGN, "bsr_w4g_proj: a must be 16-byte aligned, out 2-byte aligned");
  Device d;
  Product p;
  if ((st = device(d)) != BSR_OK) return st;
  if ((st = plan_product(p, make_args(a, m, nullptr, nullptr, w, out, m, 1, n, k), nullptr, d)) != BSR_OK) return st;
  return run_product(p, d, stream);
}

size_t bsr_w4g_proj_grouped_scratch_bytes(int64_t r, int64_t experts, int64_t k) {
  if (r <= 0 || !dim_ok(r) || experts < 1 || experts > bsr::kRouteMaxExperts || k <= 0 || !dim_ok(k) ||
      few_rows(r, experts))
    return 0;
  return align256((size_t)r * (size_t)k * 2);
}

bsr_status bsr_w4g_proj_grouped(const uint16_t* a, int64_t a_rows, const int32_t* offsets, const int32_t* rows,
                                const bsr_w4g_weight* w, uint16_t* out, int64_t r, int64_t experts, int64_t n,
                                int64_t k, void* scratch, size_t scratch_bytes, void* stream) {
  bsr_status st = check_format(w, "bsr_w4g_proj_grouped", k);
  if (st != BSR_OK) return st;
  if (!dim_ok(a_rows) || !dim_ok(r) || !dim_ok(n) || !dim_ok(k) || experts < 1 || experts > bsr::kRouteMaxExperts ||
      (n > 0 && experts > BSR_W4G_MAX_DIM / n))
    return report(BSR_EINVAL,
                  "bsr_w4g_proj_grouped: dimension out of range (a_rows=%lld r=%lld experts=%lld n=%lld k=%lld; "
                  "experts <= %d, experts * n <= 2^31 - 256)",
                  (long long)a_rows, (long long)r, (long long)experts, (long long)n, (long long)k,
                  bsr::kRouteMaxExperts);
  if (r == 0 || n == 0) return ok();
  if (!a || !offsets || !out) return report(BSR_EINVAL, "bsr_w4g_proj_grouped: null pointer");
  if (!rows && a_rows < r)
    return report(BSR_EINVAL, "bsr_w4g_proj_grouped: a has %lld rows, %lld are needed without a row index",
                  (long long)a_rows, (long long)r);
  if ((st = check_weight(w, "bsr_w4g_proj_grouped")) != BSR_OK) return st;
  if (!aligned(a, 16) || !aligned(out, 2) || !aligned(offsets, 4) || !aligned(rows, 4))
    return report(BSR_EALIGN, "bsr_w4g_proj_grouped: a must be 16-byte aligned, offsets and rows 4-byte, out 2-byte");
  const size_t need = rows ? bsr_w4g_proj_grouped_scratch_bytes(r, experts, k) : 0;
  if (need && (!scratch || scratch_bytes < need))
    return report(BSR_ESCRATCH, "scratch of %zu bytes needed, %zu given", need, scratch ? scratch_bytes : (size_t)0);
  if (need && !aligned(scratch, 256)) return report(BSR_EALIGN, "scratch must be 256-byte aligned");
  Device d;
  Product p;
  if ((st = device(d)) != BSR_OK) return st;
  uint16_t* ordered = static_cast<uint16_t*>(scratch);
  if ((st = plan_product(p, make_args(a, a_rows, offsets, rows, w, out, r, experts, n, k), ordered, d)) != BSR_OK)
    return st;
  if (p.gather && (st = cuda_status(bsr::launch_w4g_gather(a, a_rows, rows, offsets, (int)experts, ordered, r, (int)k,
                                                           as_stream(stream), d.num_sms),
                                    "row gather launch")) != BSR_OK)
    return st;
  return run_product(p, d, stream);
}

size_t bsr_moe_route_scratch_bytes(int64_t tokens, int64_t experts) {
  if (tokens <= 0 || experts < 1 || experts > bsr::kRouteMaxExperts) return 0;
  return bsr::route_scratch_bytes(tokens, (int)experts);
}

bsr_status bsr_moe_route(const void* logits, int logits_type, int64_t tokens, int64_t experts, int64_t top_k,
                         unsigned flags, int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos,
                         void* scratch, size_t scratch_bytes, void* stream) {
  bsr_status st = check_route_dims("bsr_moe_route", tokens, experts, top_k);
  if (st != BSR_OK) return st;
  if (tokens > 0) {
    if ((st = check_logits("bsr_moe_route", logits, logits_type, flags)) != BSR_OK) return st;
    if (!ids || !weights || !rows || !pos) return report(BSR_EINVAL, "bsr_moe_route: null pointer");
  }
  if (!offsets) return report(BSR_EINVAL, "bsr_moe_route: null offsets");
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4))
    return report(BSR_EALIGN, "bsr_moe_route: outputs must be 4-byte aligned");
  const size_t need = bsr_moe_route_scratch_bytes(tokens, experts);
  if (need && (!scratch || scratch_bytes < need))
    return report(BSR_ESCRATCH, "scratch of %zu bytes needed, %zu given", need, scratch ? scratch_bytes : (size_t)0);
  if (need && !aligned(scratch, 4)) return report(BSR_EALIGN, "bsr_moe_route: scratch must be 4-byte aligned");
  Device d;
  if ((st = device(d)) != BSR_OK) return st;
  return cuda_status(bsr::launch_route(logits, logits_type == BSR_MOE_LOGITS_BF16, tokens, (int)experts, (int)top_k,
                                       (flags & BSR_MOE_RENORMALIZE) != 0, ids, weights, offsets, rows, pos, scratch,
                                       d.smem_optin, as_stream(stream)),
                     "route launch");
}

bsr_status bsr_moe_combine(const uint16_t* y, int64_t y_rows, const int32_t* pos, const float* weights,
                           const uint16_t* residual, uint16_t* out, int64_t tokens, int64_t top_k, int64_t n,
                           void* stream) {
  if (!dim_ok(y_rows) || !dim_ok(n) || tokens < 0 || top_k < 1 || top_k > bsr::kRouteMaxTopK ||
      tokens > BSR_W4G_MAX_DIM / top_k)
    return report(BSR_EINVAL, "bsr_moe_combine: dimension out of range (y_rows=%lld tokens=%lld top_k=%lld n=%lld)",
                  (long long)y_rows, (long long)tokens, (long long)top_k, (long long)n);
  if (tokens == 0 || n == 0) return ok();
  if ((!y && y_rows > 0) || !pos || !weights || !out) return report(BSR_EINVAL, "bsr_moe_combine: null pointer");
  if (!aligned(y, 2) || !aligned(pos, 4) || !aligned(weights, 4) || !aligned(residual, 2) || !aligned(out, 2))
    return report(BSR_EALIGN, "bsr_moe_combine: pointers must be aligned to their types");
  Device d;
  bsr_status st = device(d);
  if (st != BSR_OK) return st;
  return cuda_status(bsr::launch_combine(y, y_rows, pos, weights, residual, out, tokens, (int)top_k, (int)n,
                                         as_stream(stream), d.num_sms),
                     "combine launch");
}

size_t bsr_w4g_moe_mlp_scratch_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t inner, int64_t k) {
  if (tokens <= 0 || experts < 1 || experts > bsr::kRouteMaxExperts || top_k < 1 || top_k > experts ||
      top_k > bsr::kRouteMaxTopK || tokens > BSR_W4G_MAX_DIM / top_k || !dim_ok(inner) || !dim_ok(k) || inner == 0 ||
      k == 0 || !mlp_fits(tokens, top_k, inner, k))
    return 0;
  return mlp_layout(tokens, experts, top_k, inner, k).total;
}

bsr_status bsr_w4g_moe_mlp(const uint16_t* x, const void* logits, int logits_type, const bsr_w4g_weight* gate,
                           const bsr_w4g_weight* up, const bsr_w4g_weight* down, const uint16_t* residual,
                           uint16_t* out, int64_t tokens, int64_t experts, int64_t top_k, unsigned flags,
                           int64_t inner, int64_t k, void* scratch, size_t scratch_bytes, void* stream) {
  static const char* const who = "bsr_w4g_moe_mlp";
  bsr_status st = check_route_dims(who, tokens, experts, top_k);
  if (st != BSR_OK) return st;
  if ((st = check_format(gate, who, k)) != BSR_OK || (st = check_format(up, who, k)) != BSR_OK ||
      (st = check_format(down, who, inner)) != BSR_OK)
    return st;
  if (!dim_ok(inner) || !dim_ok(k) || experts > BSR_W4G_MAX_DIM / inner || experts > BSR_W4G_MAX_DIM / k)
    return report(BSR_EINVAL, "%s: dimension out of range (inner=%lld k=%lld; experts times each <= 2^31 - 256)", who,
                  (long long)inner, (long long)k);
  if (!mlp_fits(tokens, top_k, inner, k))
    return report(BSR_EINVAL, "%s: scratch of 2^62 bytes or more (tokens=%lld top_k=%lld inner=%lld k=%lld)", who,
                  (long long)tokens, (long long)top_k, (long long)inner, (long long)k);
  if (tokens == 0) return ok();
  if ((st = check_logits(who, logits, logits_type, flags)) != BSR_OK) return st;
  if (!x || !out) return report(BSR_EINVAL, "%s: null pointer", who);
  if ((st = check_weight(gate, who)) != BSR_OK || (st = check_weight(up, who)) != BSR_OK ||
      (st = check_weight(down, who)) != BSR_OK)
    return st;
  if (!aligned(x, 16) || !aligned(residual, 2) || !aligned(out, 2))
    return report(BSR_EALIGN, "%s: x must be 16-byte aligned, residual and out 2-byte aligned", who);
  const MlpLayout L = mlp_layout(tokens, experts, top_k, inner, k);
  if (!scratch || scratch_bytes < L.total)
    return report(BSR_ESCRATCH, "scratch of %zu bytes needed, %zu given", L.total, scratch ? scratch_bytes : (size_t)0);
  if (!aligned(scratch, 256)) return report(BSR_EALIGN, "scratch must be 256-byte aligned");
  Device d;
  if ((st = device(d)) != BSR_OK) return st;
  const int64_t pairs = tokens * top_k;
  uint8_t* s = static_cast<uint8_t*>(scratch);
  int32_t* ids = reinterpret_cast<int32_t*>(s + L.ids);
  float* weights = reinterpret_cast<float*>(s + L.weights);
  int32_t* offsets = reinterpret_cast<int32_t*>(s + L.offsets);
  int32_t* rows = reinterpret_cast<int32_t*>(s + L.rows);
  int32_t* pos = reinterpret_cast<int32_t*>(s + L.pos);
  uint16_t* g = reinterpret_cast<uint16_t*>(s + L.gate);
  uint16_t* u = reinterpret_cast<uint16_t*>(s + L.up);
  uint16_t* h = reinterpret_cast<uint16_t*>(s + L.hidden);
  uint16_t* y = reinterpret_cast<uint16_t*>(s + L.down);
  uint16_t* ordered = reinterpret_cast<uint16_t*>(s + L.ordered);
  Product pg, pu, pd;
  if ((st = plan_product(pg, make_args(x, tokens, offsets, rows, gate, g, pairs, experts, inner, k), ordered, d)) !=
          BSR_OK ||
      (st = plan_product(pu, make_args(x, tokens, offsets, rows, up, u, pairs, experts, inner, k), ordered, d)) !=
          BSR_OK ||
      (st = plan_product(pd, make_args(h, pairs, offsets, nullptr, down, y, pairs, experts, k, inner), nullptr, d)) !=
          BSR_OK)
    return st;
  const bool gather = pg.gather || pu.gather;  // once for both
  if ((st = bsr_moe_route(logits, logits_type, tokens, experts, top_k, flags, ids, weights, offsets, rows, pos,
                          s + L.route, L.ordered - L.route, stream)) != BSR_OK)
    return st;
  if (gather && (st = cuda_status(bsr::launch_w4g_gather(x, tokens, rows, offsets, (int)experts, ordered, pairs, (int)k,
                                                         as_stream(stream), d.num_sms),
                                  "row gather launch")) != BSR_OK)
    return st;
  if ((st = run_product(pg, d, stream)) != BSR_OK || (st = run_product(pu, d, stream)) != BSR_OK) return st;
  if ((st = cuda_status(bsr::launch_silu_mul(g, u, h, (int)pairs, (int)inner, as_stream(stream), d.num_sms),
                        "silu_mul launch")) != BSR_OK)
    return st;
  if ((st = run_product(pd, d, stream)) != BSR_OK) return st;
  return bsr_moe_combine(y, pairs, pos, weights, residual, out, tokens, top_k, k, stream);
}

}  // extern "C"
