// C ABI of the operators around the expert layer (include/qmoe.h, second
// part): argument checks, then one or two launches on the caller's stream.
// They keep no state between calls but the last message of a thread and one
// device status word, and allocate nothing.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "qmoe_ops.cuh"

using namespace qmoe;

namespace {

// Set by a bounded wait that ran out (qmoe_mx4_matmul), read and cleared by
// qmoe_op_poll_status.
__device__ int g_op_status;

thread_local char t_err[256] = "";
std::atomic<long long> g_wait_limit{0};
std::atomic<int> g_inject_stall{0};
constexpr long long kDefaultWaitLimit = 1LL << 21;   // parked polls: about two seconds

qmoe_status fail(qmoe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(t_err, sizeof t_err, fmt, ap);
  va_end(ap);
  return st;
}
qmoe_status done(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return QMOE_OK;
  cudaGetLastError();   // clear a launch error
  return fail(e == cudaErrorMemoryAllocation ? QMOE_ERR_OOM : QMOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define OP_CHECK(cond, ...) \
  do {                      \
    if (!(cond)) return fail(QMOE_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)
#define OP_SUPPORTED(cond, ...) \
  do {                          \
    if (!(cond)) return fail(QMOE_ERR_UNSUPPORTED, __VA_ARGS__); \
  } while (0)

#define OP_TRY(call)                    \
  do {                                  \
    const qmoe_status st_ = (call);     \
    if (st_ != QMOE_OK) return st_;     \
  } while (0)

// Every address is a multiple of the size of what it points to (null is one).
struct Address {
  const void* p;
  int bytes;
  const char* name;
};
qmoe_status check_addresses(std::initializer_list<Address> all) {
  for (const Address& a : all)
    OP_CHECK((reinterpret_cast<uintptr_t>(a.p) & (uintptr_t)(a.bytes - 1)) == 0, "%s is not aligned to %d bytes", a.name, a.bytes);
  return QMOE_OK;
}

bool dtype_ok(int d) { return d == QMOE_F32 || d == QMOE_F16 || d == QMOE_BF16; }

// Shapes every routed operator shares.
qmoe_status check_routes(int64_t T, int k, int E) {
  OP_CHECK(T >= 0, "num_tokens %lld is negative", (long long)T);
  OP_CHECK(k >= 1, "top_k %d is not positive", k);
  OP_CHECK(E >= 1, "experts %d is not positive", E);
  OP_SUPPORTED(E <= kSortMaxExperts, "experts %d: at most %d", E, kSortMaxExperts);
  OP_CHECK(T <= (INT_MAX - 1) / k, "num_tokens %lld x top_k %d does not fit 31 bits", (long long)T, k);
  return QMOE_OK;
}
qmoe_status check_rows(int64_t H, int64_t ld, int dtype) {
  OP_CHECK(dtype_ok(dtype), "dtype %d is not QMOE_F32, QMOE_F16 or QMOE_BF16", dtype);
  OP_CHECK(H >= 1 && H <= (1 << 30), "row length %lld is out of range", (long long)H);
  OP_CHECK(ld >= H, "row stride %lld is below the row length %lld", (long long)ld, (long long)H);
  return QMOE_OK;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

const char* qmoe_op_last_error(void) { return t_err; }

qmoe_status qmoe_op_set_wait_limit(int64_t iterations) {
  OP_CHECK(iterations >= 0, "wait limit %lld is negative", (long long)iterations);
  g_wait_limit.store(iterations);
  return QMOE_OK;
}

qmoe_status qmoe_op_debug_inject_stall(int enable) {
  g_inject_stall.store(enable ? 1 : 0);
  return QMOE_OK;
}

qmoe_status qmoe_op_poll_status(void) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return done(e, "synchronise");
  int st = 0;
  e = cudaMemcpyFromSymbol(&st, g_op_status, sizeof st);
  if (e != cudaSuccess) return done(e, "read the status word");
  if (st == DEV_OK) return QMOE_OK;
  const int zero = 0;
  e = cudaMemcpyToSymbol(g_op_status, &zero, sizeof zero);
  if (e != cudaSuccess) return done(e, "clear the status word");
  return fail(QMOE_ERR_TIMEOUT, "a bounded device-side wait ran out");
}

qmoe_status qmoe_expert_sort(const void* ids_dev, int id_bytes, int64_t ld_ids, int64_t num_tokens, int top_k, int experts,
                             int32_t* perm_dev, int32_t* pos_dev, int32_t* offsets_dev, void* stream) {
  OP_TRY(check_routes(num_tokens, top_k, experts));
  OP_CHECK(id_bytes == 4 || id_bytes == 8, "id_bytes %d is not 4 or 8", id_bytes);
  OP_CHECK(offsets_dev, "offsets is null");
  if (num_tokens == 0)
    return done(cudaMemsetAsync(offsets_dev, 0, ((size_t)experts + 1) * sizeof(int32_t), as_stream(stream)), "clear offsets");
  OP_CHECK(ids_dev && perm_dev && pos_dev, "ids, perm or pos is null");
  OP_TRY(check_addresses({{ids_dev, id_bytes, "ids"}, {perm_dev, 4, "perm"}, {pos_dev, 4, "pos"}, {offsets_dev, 4, "offsets"}}));
  OP_CHECK(ld_ids >= top_k, "row stride %lld of ids is below top_k %d", (long long)ld_ids, top_k);
  SortArgs a{};
  a.ids = ids_dev;
  a.id_bytes = id_bytes;
  a.ld_ids = ld_ids;
  a.R = num_tokens * top_k;
  a.k = top_k;
  a.E = experts;
  a.perm = perm_dev;
  a.pos = pos_dev;
  a.offsets = offsets_dev;
  return done(launch_expert_sort(a, as_stream(stream)), "expert sort");
}

qmoe_status qmoe_dispatch(const void* x_dev, int64_t ld_x, const int32_t* pos_dev, const int32_t* offsets_dev,
                          int64_t num_tokens, int top_k, int experts, int64_t hidden, int dtype, void* xs_dev, void* stream) {
  OP_TRY(check_routes(num_tokens, top_k, experts));
  OP_TRY(check_rows(hidden, ld_x, dtype));
  if (num_tokens == 0) return QMOE_OK;
  OP_CHECK(x_dev && pos_dev && offsets_dev && xs_dev, "x, pos, offsets or xs is null");
  const int size = dtype_size(dtype);
  OP_TRY(check_addresses({{x_dev, size, "x"}, {pos_dev, 4, "pos"}, {offsets_dev, 4, "offsets"}, {xs_dev, size, "xs"}}));
  RowsArgs a{};
  a.src = x_dev;
  a.ld_src = ld_x;
  a.pos = pos_dev;
  a.offsets = offsets_dev;
  a.T = num_tokens;
  a.H = hidden;
  a.k = top_k;
  a.E = experts;
  a.dtype = dtype;
  a.dst = xs_dev;
  return done(launch_dispatch(a, as_stream(stream)), "dispatch");
}

qmoe_status qmoe_combine(const void* y_dev, int64_t ld_y, const float* weights_dev, const int32_t* pos_dev,
                         int64_t num_tokens, int top_k, int64_t hidden, int dtype, void* out_dev, void* stream) {
  OP_TRY(check_routes(num_tokens, top_k, 1));
  OP_TRY(check_rows(hidden, ld_y, dtype));
  if (num_tokens == 0) return QMOE_OK;
  OP_CHECK(y_dev && pos_dev && out_dev, "y, pos or out is null");
  const int size = dtype_size(dtype);
  OP_TRY(check_addresses({{y_dev, size, "y"}, {weights_dev, 4, "weights"}, {pos_dev, 4, "pos"}, {out_dev, size, "out"}}));
  RowsArgs a{};
  a.src = y_dev;
  a.ld_src = ld_y;
  a.w = weights_dev;
  a.pos = pos_dev;
  a.T = num_tokens;
  a.H = hidden;
  a.k = top_k;
  a.dtype = dtype;
  a.dst = out_dev;
  return done(launch_combine(a, as_stream(stream)), "combine");
}

qmoe_status qmoe_dispatch_grad(const void* dxs_dev, int64_t ld_dxs, const int32_t* pos_dev, int64_t num_tokens, int top_k,
                               int64_t hidden, int dtype, void* dx_dev, void* stream) {
  return qmoe_combine(dxs_dev, ld_dxs, nullptr, pos_dev, num_tokens, top_k, hidden, dtype, dx_dev, stream);
}

qmoe_status qmoe_combine_grad(const void* dout_dev, int64_t ld_dout, const void* y_dev, int64_t ld_y,
                              const float* weights_dev, const int32_t* pos_dev, const int32_t* offsets_dev,
                              int64_t num_tokens, int top_k, int experts, int64_t hidden, int dtype, void* dy_dev,
                              float* dweights_dev, void* stream) {
  OP_TRY(check_routes(num_tokens, top_k, experts));
  OP_TRY(check_rows(hidden, ld_dout, dtype));
  if (dweights_dev) OP_TRY(check_rows(hidden, ld_y, dtype));
  if (num_tokens == 0 || (!dy_dev && !dweights_dev)) return QMOE_OK;
  OP_CHECK(dout_dev && pos_dev, "dout or pos is null");
  OP_CHECK(!dy_dev || offsets_dev, "dy needs offsets");
  OP_CHECK(!dweights_dev || y_dev, "dweights needs y");
  const int size = dtype_size(dtype);
  OP_TRY(check_addresses({{dout_dev, size, "dout"}, {dweights_dev ? y_dev : nullptr, size, "y"}, {weights_dev, 4, "weights"},
                          {pos_dev, 4, "pos"}, {offsets_dev, 4, "offsets"}, {dy_dev, size, "dy"}, {dweights_dev, 4, "dweights"}}));
  RowsArgs a{};
  a.src = dout_dev;
  a.ld_src = ld_dout;
  a.y = dweights_dev ? y_dev : nullptr;
  a.ld_y = ld_y;
  a.w = weights_dev;
  a.pos = pos_dev;
  a.offsets = offsets_dev;
  a.T = num_tokens;
  a.H = hidden;
  a.k = top_k;
  a.E = experts;
  a.dtype = dtype;
  a.dst = dy_dev;
  a.dw = dweights_dev;
  return done(launch_combine_grad(a, as_stream(stream)), "combine gradient");
}

qmoe_status qmoe_mx4_quantize(const void* x_dev, int64_t ld_x, int64_t rows, int64_t cols, int dtype, int activation,
                              const int32_t* pos_dev, const int32_t* offsets_dev, int top_k, int experts,
                              int64_t panel_rows, uint8_t* codes_dev, uint8_t* scales_dev, void* stream) {
  OP_CHECK(rows >= 0, "rows %lld is negative", (long long)rows);
  OP_CHECK(activation == QMOE_ACT_NONE || activation == QMOE_ACT_SWIGLU || activation == QMOE_ACT_GEGLU_TANH,
           "activation %d is not QMOE_ACT_NONE or a gated one", activation);
  OP_CHECK(cols >= 1 && cols <= (1 << 29), "cols %lld is out of range", (long long)cols);
  OP_TRY(check_rows(activation == QMOE_ACT_NONE ? cols : 2 * cols, ld_x, dtype));
  int64_t out_rows = rows;
  if (pos_dev) {
    OP_TRY(check_routes(rows, top_k, experts));
    OP_CHECK(offsets_dev, "offsets is null beside pos");
    out_rows = rows * top_k;
    OP_CHECK(panel_rows == out_rows, "panel_rows %lld: with pos the output is one panel of %lld rows", (long long)panel_rows,
             (long long)out_rows);
  }
  OP_CHECK(panel_rows >= 1 || out_rows == 0, "panel_rows %lld is not positive", (long long)panel_rows);
  OP_CHECK(out_rows == 0 || out_rows % panel_rows == 0, "panel_rows %lld does not divide the %lld rows",
           (long long)panel_rows, (long long)out_rows);
  if (out_rows == 0) return QMOE_OK;
  OP_CHECK(x_dev && codes_dev && scales_dev, "x, codes or scales is null");
  OP_TRY(check_addresses({{x_dev, dtype_size(dtype), "x"}, {pos_dev, 4, "pos"}, {offsets_dev, 4, "offsets"},
                          {codes_dev, 16, "codes"}, {scales_dev, 4, "scales"}}));
  Mx4QuantArgs a{};
  a.x = x_dev;
  a.ld_x = ld_x;
  a.rows = rows;
  a.cols = cols;
  a.dtype = dtype;
  a.act = ActParams{activation, 1.f, 0.f, INFINITY};
  a.pos = pos_dev;
  a.offsets = offsets_dev;
  a.k = top_k;
  a.E = experts;
  a.panel = panel_rows;
  a.codes = codes_dev;
  a.scales = scales_dev;
  return done(launch_mx4_quantize(a, as_stream(stream)), "mx4 quantize");
}

qmoe_status qmoe_mx4_dequantize(const uint8_t* codes_dev, const uint8_t* scales_dev, int64_t rows, int64_t cols,
                                int64_t panel_rows, int dtype, void* out_dev, int64_t ld_out, void* stream) {
  OP_CHECK(rows >= 0, "rows %lld is negative", (long long)rows);
  OP_TRY(check_rows(cols, ld_out, dtype));
  OP_CHECK(rows == 0 || (panel_rows >= 1 && rows % panel_rows == 0), "panel_rows %lld does not divide the %lld rows",
           (long long)panel_rows, (long long)rows);
  if (rows == 0) return QMOE_OK;
  OP_CHECK(codes_dev && scales_dev && out_dev, "codes, scales or out is null");
  OP_TRY(check_addresses({{codes_dev, 4, "codes"}, {out_dev, dtype_size(dtype), "out"}}));
  Mx4DequantArgs a{};
  a.codes = codes_dev;
  a.scales = scales_dev;
  a.rows = rows;
  a.cols = cols;
  a.panel = panel_rows;
  a.dtype = dtype;
  a.out = out_dev;
  a.ld_out = ld_out;
  return done(launch_mx4_dequantize(a, as_stream(stream)), "mx4 dequantize");
}

qmoe_status qmoe_mx4_matmul(const uint8_t* a_codes_dev, const uint8_t* a_scales_dev, int64_t rows,
                            const uint8_t* w_codes_dev, const uint8_t* w_scales_dev, const int32_t* offsets_dev,
                            int experts, int64_t n, int64_t k, int out_dtype, void* out_dev, int64_t ld_out, void* stream) {
  // a tile's rows, of either operand, may reach past the last one by less than this
  constexpr int reach = 256;
  OP_CHECK(rows >= 0, "rows %lld is negative", (long long)rows);
  OP_CHECK(rows < INT_MAX - reach, "rows %lld do not fit 31 bits", (long long)rows);
  OP_CHECK(experts >= 1, "experts %d is not positive", experts);
  OP_SUPPORTED(experts <= kSortMaxExperts, "experts %d: at most %d", experts, kSortMaxExperts);
  OP_CHECK(offsets_dev || experts == 1, "%d experts need offsets", experts);
  OP_TRY(check_rows(n, ld_out, out_dtype));
  OP_CHECK(k >= 1 && k < (1LL << 30), "reduction length %lld is out of range", (long long)k);
  OP_CHECK(n < (INT_MAX - reach) / experts, "%d experts of %lld rows do not fit 31 bits", experts, (long long)n);
  if (rows == 0) return QMOE_OK;
  OP_CHECK(a_codes_dev && a_scales_dev && w_codes_dev && w_scales_dev && out_dev, "an operand or out is null");
  OP_TRY(check_addresses({{a_codes_dev, 16, "a's codes"}, {a_scales_dev, 4, "a's scales"}, {w_codes_dev, 16, "w's codes"},
                          {w_scales_dev, 4, "w's scales"}, {offsets_dev, 4, "offsets"}, {out_dev, dtype_size(out_dtype), "out"}}));
  Mx4MatmulArgs a{};
  a.a_codes = a_codes_dev;
  a.a_scales = a_scales_dev;
  a.w_codes = w_codes_dev;
  a.w_scales = w_scales_dev;
  a.offsets = offsets_dev;
  a.R = rows;
  a.E = experts;
  a.N = (int)n;
  a.K = (int)k;
  a.out_dtype = out_dtype;
  a.out = out_dev;
  a.ld_out = ld_out;
  void* status = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&status, g_op_status);
  if (e != cudaSuccess) return done(e, "look up the status word");
  const long long limit = g_wait_limit.load();
  a.wait = WaitCfg{static_cast<int*>(status), limit ? limit : kDefaultWaitLimit};
  return done(launch_mx4_matmul(a, g_inject_stall.load(), as_stream(stream)), "mx4 matmul");
}

static qmoe_status norm_args(NormArgs& a, const void* x, int64_t ld_x, const void* o, int64_t ld_o, const void* gate,
                             int gate_kind, int64_t ld_gate, const void* w_post, const void* w_pre, float residual_scale,
                             float eps, int64_t T, int64_t H, int dtype) {
  OP_CHECK(T >= 0 && T < INT_MAX, "num_tokens %lld is out of range", (long long)T);
  OP_TRY(check_rows(H, ld_x, dtype));
  OP_SUPPORTED(H <= kNormMaxWidth, "row length %lld: at most %lld", (long long)H, (long long)kNormMaxWidth);
  OP_CHECK(gate_kind >= QMOE_GATE_NONE && gate_kind <= QMOE_GATE_FULL, "gate_kind %d is unknown", gate_kind);
  OP_CHECK(std::isfinite(eps) && eps >= 0.f, "eps must be finite and not negative");
  OP_CHECK(std::isfinite(residual_scale), "residual_scale must be finite");
  OP_CHECK(x || T == 0, "x is null");
  OP_CHECK(o || T == 0 || (!w_post && gate_kind == QMOE_GATE_NONE), "w_post and gate need o");
  OP_CHECK(!o || ld_o >= H, "row stride %lld of o is below the row length %lld", (long long)ld_o, (long long)H);
  // without tokens a gate of one or more values a token is empty, and may be null
  const bool empty = T == 0 && (gate_kind == QMOE_GATE_TOKEN || gate_kind == QMOE_GATE_FULL);
  OP_CHECK((gate != nullptr) == (gate_kind != QMOE_GATE_NONE) || empty, "gate and gate_kind disagree");
  OP_CHECK(gate_kind != QMOE_GATE_FULL || ld_gate >= H, "row stride %lld of gate is below the row length %lld",
           (long long)ld_gate, (long long)H);
  const int size = dtype_size(dtype);
  OP_TRY(check_addresses({{x, size, "x"}, {o, size, "o"}, {gate, size, "gate"}, {w_post, size, "w_post"}, {w_pre, size, "w_pre"}}));
  a.x = x;
  a.ld_x = ld_x;
  a.o = o;
  a.ld_o = ld_o;
  a.gate = gate;
  a.gate_kind = gate_kind;
  a.ld_gate = ld_gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.residual_scale = residual_scale;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.dtype = dtype;
  return QMOE_OK;
}

qmoe_status qmoe_block_norm(const void* x_dev, int64_t ld_x, const void* o_dev, int64_t ld_o, const void* gate_dev,
                            int gate_kind, int64_t ld_gate, const void* w_post_dev, const void* w_pre_dev,
                            float residual_scale, float eps, int64_t num_tokens, int64_t hidden, int dtype, void* r_dev,
                            void* h_dev, float* rstd_post_dev, float* rstd_pre_dev, void* stream) {
  NormArgs a{};
  OP_TRY(norm_args(a, x_dev, ld_x, o_dev, ld_o, gate_dev, gate_kind, ld_gate, w_post_dev, w_pre_dev, residual_scale, eps,
                   num_tokens, hidden, dtype));
  OP_CHECK((w_pre_dev != nullptr) == (h_dev != nullptr) || num_tokens == 0, "w_pre and h go together");
  OP_CHECK(r_dev || h_dev || num_tokens == 0, "neither r nor h is asked for");
  if (num_tokens == 0) return QMOE_OK;
  const int size = dtype_size(dtype);
  OP_TRY(check_addresses({{r_dev, size, "r"}, {h_dev, size, "h"}, {rstd_post_dev, 4, "rstd_post"}, {rstd_pre_dev, 4, "rstd_pre"}}));
  a.r = r_dev;
  a.h = h_dev;
  a.rstd_post = w_post_dev ? rstd_post_dev : nullptr;
  a.rstd_pre = rstd_pre_dev;
  return done(launch_block_norm(a, as_stream(stream)), "block norm");
}

size_t qmoe_block_norm_grad_workspace(int64_t num_tokens, int64_t hidden, int dtype) {
  if (num_tokens < 0 || hidden < 1 || hidden > kNormMaxWidth || !dtype_ok(dtype)) return 0;
  return block_norm_grad_workspace(num_tokens, hidden, dtype);
}

qmoe_status qmoe_block_norm_grad(const void* dr_dev, int64_t ld_dr, const void* dh_dev, int64_t ld_dh, const void* x_dev,
                                 int64_t ld_x, const void* o_dev, int64_t ld_o, const void* gate_dev, int gate_kind,
                                 int64_t ld_gate, const void* w_post_dev, const void* w_pre_dev,
                                 const float* rstd_post_dev, const float* rstd_pre_dev, float residual_scale,
                                 int64_t num_tokens, int64_t hidden, int dtype, void* dx_dev, void* do_dev,
                                 void* dgate_dev, void* dw_post_dev, void* dw_pre_dev, void* workspace_dev,
                                 size_t workspace_bytes, void* stream) {
  NormArgs a{};
  OP_TRY(norm_args(a, x_dev, ld_x, o_dev, ld_o, gate_dev, gate_kind, ld_gate, w_post_dev, w_pre_dev, residual_scale, 0.f,
                   num_tokens, hidden, dtype));
  OP_CHECK(!dr_dev || ld_dr >= hidden, "row stride %lld of dr is below the row length %lld", (long long)ld_dr,
           (long long)hidden);
  OP_CHECK(!dh_dev || (w_pre_dev && ld_dh >= hidden), "dh needs w_pre and a row stride of at least the row length");
  OP_CHECK(!dw_pre_dev || w_pre_dev, "dw_pre needs w_pre");
  OP_CHECK(!dw_post_dev || w_post_dev, "dw_post needs w_post");
  OP_CHECK(!dgate_dev || gate_kind != QMOE_GATE_NONE, "dgate needs gate");
  OP_CHECK(!do_dev || o_dev || num_tokens == 0, "do needs o");
  OP_CHECK(num_tokens == 0 || (!w_post_dev || rstd_post_dev), "w_post needs rstd_post");
  OP_CHECK(num_tokens == 0 || (!w_pre_dev || rstd_pre_dev), "w_pre needs rstd_pre");
  const size_t need = block_norm_grad_workspace(num_tokens, hidden, dtype);
  OP_CHECK(workspace_bytes >= need && (workspace_dev || need == 0), "workspace of %zu bytes is below the %zu needed",
           workspace_bytes, need);
  const int size = dtype_size(dtype);
  OP_TRY(check_addresses({{dr_dev, size, "dr"}, {dh_dev, size, "dh"}, {rstd_post_dev, 4, "rstd_post"},
                          {rstd_pre_dev, 4, "rstd_pre"}, {dx_dev, size, "dx"}, {do_dev, size, "do"}, {dgate_dev, size, "dgate"},
                          {dw_post_dev, size, "dw_post"}, {dw_pre_dev, size, "dw_pre"}, {workspace_dev, 4, "workspace"}}));
  a.dr = dr_dev;
  a.ld_dr = ld_dr;
  a.dh = dh_dev;
  a.ld_dh = ld_dh;
  a.rstd_post = const_cast<float*>(rstd_post_dev);
  a.rstd_pre = const_cast<float*>(rstd_pre_dev);
  a.dx = dx_dev;
  a.d_o = do_dev;
  a.dgate = dgate_dev;
  a.dw_post = dw_post_dev;
  a.dw_pre = dw_pre_dev;
  a.partial = static_cast<float*>(workspace_dev);
  return done(launch_block_norm_grad(a, as_stream(stream)), "block norm gradient");
}

}  // extern "C"
