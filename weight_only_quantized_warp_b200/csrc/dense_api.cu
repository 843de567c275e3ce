// dense_api.cu -- C entry points of the dense operators declared in
// include/qmoe.h: argument checks, workspace layout and launch sequences.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "dense.cuh"

using namespace qmoe;

namespace {

thread_local char g_error[256] = "";

qmoe_status bad(qmoe_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof g_error, fmt, ap);
    va_end(ap);
    return s;
}

qmoe_status cuda_bad(cudaError_t e, const char* where) {
    return bad(QMOE_CUDA_ERROR, "%s: %s", where, cudaGetErrorString(e));
}

bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) & (n - 1); }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// The launches go to the current device: a tensor of another one is refused.
qmoe_status on_current_device(const void* p) {
    int dev = 0;
    cudaPointerAttributes at;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) return cuda_bad(e, "device of the output");
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
        return bad(QMOE_INVALID_ARGUMENT, "not a device pointer");
    if (at.type == cudaMemoryTypeDevice && at.device != dev)
        return bad(QMOE_INVALID_ARGUMENT, "the output is on device %d, the current device is %d", at.device, dev);
    return QMOE_OK;
}

qmoe_status check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws || misaligned(ws, 256)) return bad(QMOE_INVALID_ARGUMENT, "the workspace must be 256-byte aligned");
    if (have < need) return bad(QMOE_INVALID_ARGUMENT, "workspace too small: %zu < %zu", have, need);
    return QMOE_OK;
}

// Workspaces begin with the device status word; parts are 256-byte aligned.
struct Layout {
    size_t total = 256;
    size_t take(size_t bytes) {
        const size_t at = total;
        total += (bytes + 255) & ~size_t(255);
        return at;
    }
};

qmoe_status check_mx4_rows(const void* x, int32_t dtype, int64_t rows, int64_t K, int64_t ldx, const void* codes,
                           const void* scales) {
    if (dtype != QMOE_DTYPE_F32 && dtype != QMOE_DTYPE_BF16)
        return bad(QMOE_INVALID_ARGUMENT, "dtype must be F32 or BF16");
    if (rows < 0 || K < 32 || K % 32) return bad(QMOE_INVALID_ARGUMENT, "rows >= 0 and K a positive multiple of 32");
    if (K > kMaxDim || rows > kMaxDim || rows > (int64_t(1) << 48) / K)
        return bad(QMOE_UNSUPPORTED, "rows or K too large");
    const int per16 = dtype == QMOE_DTYPE_F32 ? 4 : 8;
    if (rows > 1 && (ldx < K || ldx % per16 || ldx > (int64_t(1) << 40) / rows))
        return bad(QMOE_INVALID_ARGUMENT, "ldx must be at least K and a multiple of 16 bytes");
    if (rows == 0) return QMOE_OK;
    if (!x || !codes || !scales) return bad(QMOE_INVALID_ARGUMENT, "x, codes and scales are required");
    if (misaligned(x, 16) || misaligned(codes, 4))
        return bad(QMOE_INVALID_ARGUMENT, "x must be 16-byte, codes 4-byte aligned");
    return QMOE_OK;
}

// Checked configuration: the gate's parameters.
qmoe_status check_ffn(const qmoe_gated_ffn_config* c, int64_t T, GateParams* g) {
    if (!c) return bad(QMOE_INVALID_ARGUMENT, "cfg is required");
    if (c->hidden_size < 1 || c->inter_size < 1 || T < 0)
        return bad(QMOE_INVALID_ARGUMENT, "hidden_size and inter_size must be positive, T >= 0");
    if (c->activation_type < QMOE_ACT_RELU || c->activation_type > QMOE_ACT_IDENTITY)
        return bad(QMOE_INVALID_ARGUMENT, "unknown activation_type");
    if (c->swiglu_fusion != 1 && c->swiglu_fusion != 2)
        return bad(QMOE_INVALID_ARGUMENT, "swiglu_fusion must be 1 or 2");
    if (c->gelu_mode != QMOE_GELU_ERF && c->gelu_mode != QMOE_GELU_TANH)
        return bad(QMOE_INVALID_ARGUMENT, "unknown gelu_mode");
    if (c->act_dtype != QMOE_DTYPE_F32 && c->act_dtype != QMOE_DTYPE_BF16)
        return bad(QMOE_INVALID_ARGUMENT, "act_dtype must be BF16");
    if (c->reserved) return bad(QMOE_INVALID_ARGUMENT, "reserved must be 0");
    if (!std::isfinite(c->activation_alpha) || !std::isfinite(c->activation_beta))
        return bad(QMOE_INVALID_ARGUMENT, "activation_alpha and activation_beta must be finite");
    if (c->act_dtype == QMOE_DTYPE_F32) return bad(QMOE_UNSUPPORTED, "fp32 activations are not built");
    if (c->hidden_size % 8 || c->inter_size % 8)
        return bad(QMOE_UNSUPPORTED, "hidden_size and inter_size must be multiples of 8");
    if (T > kMaxDim || c->hidden_size > kMaxDim / 2 || c->inter_size > kMaxDim / 2)
        return bad(QMOE_UNSUPPORTED, "T, hidden_size or inter_size too large");
    if (g) {
        const int t = c->activation_type;
        const bool swiglu = t == QMOE_ACT_SWIGLU, tanh = t == QMOE_ACT_GELU && c->gelu_mode == QMOE_GELU_TANH;
        g->mode = t == QMOE_ACT_RELU       ? kGateStep
                  : t == QMOE_ACT_IDENTITY ? kGateOne
                  : t == QMOE_ACT_GELU && !tanh ? kGateErf
                                                : kGateSigmoid;
        const float k = 1.5957691216057308f;  // 2 sqrt(2 / pi)
        g->c1 = tanh ? k : swiglu && c->activation_alpha != 0.0f ? c->activation_alpha : 1.0f;
        g->c3 = tanh ? k * 0.044715f : 0.0f;
        g->beta = swiglu ? c->activation_beta : 0.0f;
        g->limit = swiglu && c->swiglu_limit > 0.0f && std::isfinite(c->swiglu_limit) ? c->swiglu_limit : INFINITY;
    }
    return QMOE_OK;
}

struct FfnLayout : Layout {
    size_t h = 0, dgu = 0, sums = 0, part = 0;
    FfnLayout(const qmoe_gated_ffn_config& c, int64_t T, bool backward) {
        h = take(size_t(T) * c.inter_size * 2);
        if (backward) {
            dgu = take(size_t(T) * c.inter_size * 4);
            const int64_t rows = dense_sum_rows_most(T, c.inter_size, c.hidden_size);
            sums = take(size_t(rows) * c.inter_size * 8);
            part = take(colsum_bytes(rows, 2 * c.inter_size, T, c.hidden_size));
        }
    }
};

// Few rows stream the weights, more run on CTA pairs.
cudaError_t launch_rows(const DenseArgs& a, bool early, cudaStream_t st) {
    return dense_streams(a.M, a.mx4 ? a.N * (a.K / 2) : a.N * a.K * 2) ? launch_dense_stream(a, early, st)
                                                                       : launch_dense_pair(a, early, st);
}

qmoe_status check_linear_sizes(int64_t T, int64_t N, int64_t K) {
    if (T < 0 || N < 1 || K < 32 || K % 32)
        return bad(QMOE_INVALID_ARGUMENT, "T >= 0, N >= 1 and K a positive multiple of 32");
    if (T > kMaxDim || N > kMaxDim || K > kMaxDim) return bad(QMOE_UNSUPPORTED, "T, N or K too large");
    return QMOE_OK;
}

qmoe_status check_linear_tensors(const void* w_codes, const void* w_scales, const void* bias, const void* y,
                                 int32_t dtype) {
    if (!w_codes || !w_scales || !y) return bad(QMOE_INVALID_ARGUMENT, "w_codes, w_scales and y are required");
    if (misaligned(w_codes, 16) || misaligned(w_scales, 4))
        return bad(QMOE_INVALID_ARGUMENT, "codes must be 16-byte, scales 4-byte aligned");
    const int es = dtype == QMOE_DTYPE_F32 ? 4 : 2;
    if (misaligned(y, es) || misaligned(bias, es))
        return bad(QMOE_INVALID_ARGUMENT, "y and bias must be aligned to their elements");
    return QMOE_OK;
}

// Tiled scales where the product runs on CTA pairs; the rounded rows of x where
// the call rounds them (their scales by rows where the product streams).
struct LinearLayout : Layout {
    bool streams;
    size_t tiles = 0, codes = 0, scales = 0;
    LinearLayout(int64_t T, int64_t N, int64_t K, bool rows) : streams(dense_streams(T, N * (K / 2))) {
        if (!streams) tiles = take(dense_pair_workspace(T, N, K));
        if (rows) codes = take(size_t(T) * size_t(K / 2));
        if (rows) scales = streams ? take(size_t(T) * size_t(K / 32)) : codes;
    }
};

DenseArgs linear_args(int64_t T, int64_t N, int64_t K, const uint8_t* xc, const uint8_t* xs, const uint8_t* wc,
                      const uint8_t* ws, const void* bias, void* y, int32_t dtype, void* workspace,
                      const LinearLayout& l) {
    DenseArgs a{};
    a.a = {xc, xs, 0, 0};
    a.b = {wc, ws, 0, 0};
    a.M = T;
    a.N = N;
    a.K = K;
    a.mx4 = 1;
    a.epi = kEpiStore;
    a.out_f32 = dtype == QMOE_DTYPE_F32;
    a.bias = bias;
    a.out = y;
    a.status = (int32_t*)workspace;
    a.reset_status = 1;
    a.scratch = l.streams ? nullptr : (char*)workspace + l.tiles;
    return a;
}

DenseOperand rows_of(const void* p, int64_t ld) { return {p, nullptr, ld, 1}; }   // k along the row
DenseOperand cols_of(const void* p, int64_t ld) { return {p, nullptr, 1, ld}; }   // k across the rows

std::atomic<uint64_t> g_wait_limit_ns{2000000000ull};
std::atomic<int> g_withhold{0};

// Counts of expired waits (pair, stream) that a device's last report covered.
constexpr int kMaxDevices = 64;
std::mutex g_reported_mu;
uint32_t g_reported[kMaxDevices][2];

}  // namespace

namespace qmoe {
DenseWaits dense_waits() {
    return {g_wait_limit_ns.load(std::memory_order_relaxed), g_withhold.load(std::memory_order_relaxed)};
}
}  // namespace qmoe

extern "C" {

const char* qmoe_dense_last_error(void) { return g_error; }

qmoe_status qmoe_dense_read_device_status(const void* workspace, void* stream) {
    if (!workspace) return bad(QMOE_INVALID_ARGUMENT, "workspace is required");
    int32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, workspace, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_bad(e, "read_device_status");
    return v == 0 ? QMOE_OK : QMOE_TIMEOUT;
}

qmoe_status qmoe_dense_take_device_status(void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    int dev = 0;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaStreamIsCapturing(st, &cs);
    if (e != cudaSuccess) return cuda_bad(e, "take_device_status");
    if (cs != cudaStreamCaptureStatusNone)
        return bad(QMOE_INVALID_ARGUMENT, "the stream is being captured: the status is read on the host");
    if (dev >= kMaxDevices) return bad(QMOE_UNSUPPORTED, "device index above %d", kMaxDevices - 1);
    std::lock_guard<std::mutex> lock(g_reported_mu);
    uint32_t now[2] = {};
    e = dense_pair_gave_up(&now[0], st);
    if (e == cudaSuccess) e = dense_stream_gave_up(&now[1], st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_bad(e, "take_device_status");
    uint32_t* seen = g_reported[dev];
    const bool same = seen[0] == now[0] && seen[1] == now[1];
    seen[0] = now[0];
    seen[1] = now[1];
    return same ? QMOE_OK
                : bad(QMOE_TIMEOUT, "a bounded device wait of a dense call gave up since the last report: "
                                    "the results of the calls since then are undefined");
}

qmoe_status qmoe_dense_set_option(int32_t option, int64_t value) {
    if (option == QMOE_OPT_WAIT_LIMIT_NS) {
        if (value < 100000 || value > 60000000000ll)
            return bad(QMOE_INVALID_ARGUMENT, "QMOE_OPT_WAIT_LIMIT_NS must lie in [1e5, 6e10] ns");
        g_wait_limit_ns.store(uint64_t(value), std::memory_order_relaxed);
        return QMOE_OK;
    }
    if (option == QMOE_OPT_TEST_WITHHOLD) {
        if (value != 0 && value != 1) return bad(QMOE_INVALID_ARGUMENT, "QMOE_OPT_TEST_WITHHOLD must be 0 or 1");
        g_withhold.store(int(value), std::memory_order_relaxed);
        return QMOE_OK;
    }
    return bad(QMOE_INVALID_ARGUMENT, "unknown option of the dense calls");
}

qmoe_status qmoe_mx4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                              uint8_t* scales, void* stream) {
    if (qmoe_status s = check_mx4_rows(x, dtype, rows, K, ldx, codes, scales)) return s;
    if (rows == 0) return QMOE_OK;
    if (qmoe_status s = on_current_device(codes)) return s;
    const cudaError_t e = launch_mx4_quantize(x, dtype == QMOE_DTYPE_BF16, rows, K, rows > 1 ? ldx : K, codes, scales,
                                              (cudaStream_t)stream);
    return e == cudaSuccess ? QMOE_OK : cuda_bad(e, "mx4_quantize");
}

qmoe_status qmoe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* x,
                                int32_t dtype, int64_t ldx, void* stream) {
    if (qmoe_status s = check_mx4_rows(x, dtype, rows, K, ldx, codes, scales)) return s;
    if (rows == 0) return QMOE_OK;
    if (qmoe_status s = on_current_device(x)) return s;
    const cudaError_t e = launch_mx4_dequantize(codes, scales, rows, K, x, dtype == QMOE_DTYPE_BF16,
                                                rows > 1 ? ldx : K, (cudaStream_t)stream);
    return e == cudaSuccess ? QMOE_OK : cuda_bad(e, "mx4_dequantize");
}

size_t qmoe_mx4_linear_workspace_size(int64_t T, int64_t N, int64_t K) {
    return check_linear_sizes(T, N, K) ? 0 : LinearLayout(T, N, K, false).total;
}

qmoe_status qmoe_mx4_linear(int64_t T, int64_t N, int64_t K, const uint8_t* x_codes, const uint8_t* x_scales,
                            const uint8_t* w_codes, const uint8_t* w_scales, const void* bias, void* y, int32_t dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
    if (qmoe_status s = check_linear_sizes(T, N, K)) return s;
    if (dtype != QMOE_DTYPE_F32 && dtype != QMOE_DTYPE_BF16)
        return bad(QMOE_INVALID_ARGUMENT, "dtype must be F32 or BF16");
    if (T == 0) return QMOE_OK;
    if (!x_codes || !x_scales || misaligned(x_codes, 16) || misaligned(x_scales, 4))
        return bad(QMOE_INVALID_ARGUMENT, "x_codes (16-byte) and x_scales (4-byte aligned) are required");
    if (qmoe_status s = check_linear_tensors(w_codes, w_scales, bias, y, dtype)) return s;
    const LinearLayout l(T, N, K, false);
    if (qmoe_status s = check_workspace(workspace, workspace_bytes, l.total)) return s;
    if (qmoe_status s = on_current_device(y)) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const DenseArgs a = linear_args(T, N, K, x_codes, x_scales, w_codes, w_scales, bias, y, dtype, workspace, l);
    cudaError_t e = cudaSuccess;
    if (a.scratch) {
        ScaleTiles ta, tb;
        dense_pair_tiles(T, N, K, a.scratch, &ta, &tb);
        ta.s = x_scales;
        tb.s = w_scales;
        e = launch_mx4_tile_scales(ta, tb, K, st);
    }
    if (e == cudaSuccess) e = launch_rows(a, false, st);
    return e == cudaSuccess ? QMOE_OK : cuda_bad(e, "mx4_linear");
}

size_t qmoe_mx4_linear_rows_workspace_size(int64_t T, int64_t N, int64_t K) {
    return check_linear_sizes(T, N, K) ? 0 : LinearLayout(T, N, K, true).total;
}

qmoe_status qmoe_mx4_linear_rows(int64_t T, int64_t N, int64_t K, const void* x, int64_t ldx, const uint8_t* w_codes,
                                 const uint8_t* w_scales, const void* bias, void* y, int32_t dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (qmoe_status s = check_linear_sizes(T, N, K)) return s;
    const LinearLayout l(T, N, K, true);
    uint8_t* codes = (uint8_t*)workspace + l.codes;
    uint8_t* scales = (uint8_t*)workspace + l.scales;
    if (T > 0)
        if (qmoe_status s = check_workspace(workspace, workspace_bytes, l.total)) return s;
    if (qmoe_status s = check_mx4_rows(x, dtype, T, K, ldx, codes, scales)) return s;
    if (T == 0) return QMOE_OK;
    if (qmoe_status s = check_linear_tensors(w_codes, w_scales, bias, y, dtype)) return s;
    if (qmoe_status s = on_current_device(y)) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const int bf16 = dtype == QMOE_DTYPE_BF16;
    const int64_t ld = T > 1 ? ldx : K;
    const DenseArgs a = linear_args(T, N, K, codes, scales, w_codes, w_scales, bias, y, dtype, workspace, l);
    cudaError_t e;
    if (a.scratch) {
        ScaleTiles ta, tb;
        dense_pair_tiles(T, N, K, a.scratch, &ta, &tb);
        tb.s = w_scales;
        e = launch_mx4_quantize_tiled(x, bf16, T, K, ld, codes, ta, tb, st);
    } else {
        e = launch_mx4_quantize(x, bf16, T, K, ld, codes, scales, st);
    }
    if (e == cudaSuccess) e = launch_rows(a, true, st);  // the rounding wrote none of the weights
    return e == cudaSuccess ? QMOE_OK : cuda_bad(e, "mx4_linear_rows");
}

size_t qmoe_gated_ffn_workspace_size(const qmoe_gated_ffn_config* cfg, int64_t T, int32_t backward) {
    if (check_ffn(cfg, T, nullptr)) return 0;
    return FfnLayout(*cfg, T, backward != 0).total;
}

qmoe_status qmoe_gated_ffn_forward(const qmoe_gated_ffn_config* cfg, int64_t T, const void* x, const void* w1,
                                   const void* b1, const void* w2, const void* b2, float* gu, void* y,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    GateParams gate;
    if (qmoe_status s = check_ffn(cfg, T, &gate)) return s;
    if (T == 0) return QMOE_OK;
    if (!x || !w1 || !w2 || !y) return bad(QMOE_INVALID_ARGUMENT, "x, w1, w2 and y are required");
    if (misaligned(x, 16) || misaligned(w1, 16) || misaligned(w2, 16) || misaligned(y, 16) || misaligned(gu, 16) ||
        misaligned(b1, 2) || misaligned(b2, 2))
        return bad(QMOE_INVALID_ARGUMENT, "tensors must be 16-byte, biases 2-byte aligned");
    const FfnLayout l(*cfg, T, false);
    if (qmoe_status s = check_workspace(workspace, workspace_bytes, l.total)) return s;
    if (qmoe_status s = on_current_device(y)) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t H = cfg->hidden_size, I = cfg->inter_size;
    void* h = (char*)workspace + l.h;
    DenseArgs a{};
    a.a = rows_of(x, H);
    a.b = rows_of(w1, H);
    a.M = T;
    a.N = 2 * I;
    a.K = H;
    a.epi = kEpiGate;
    a.bias = b1;
    a.out = h;
    a.gu = gu;
    a.gate = gate;
    a.interleaved = cfg->swiglu_fusion == 1;
    a.status = (int32_t*)workspace;
    a.reset_status = 1;
    cudaError_t e = launch_rows(a, false, st);
    DenseArgs d{};
    d.a = rows_of(h, I);
    d.b = rows_of(w2, I);
    d.M = T;
    d.N = H;
    d.K = I;
    d.epi = kEpiStore;
    d.bias = b2;
    d.out = y;
    d.status = (int32_t*)workspace;
    if (e == cudaSuccess) e = launch_rows(d, true, st);
    return e == cudaSuccess ? QMOE_OK : cuda_bad(e, "gated_ffn_forward");
}

qmoe_status qmoe_gated_ffn_backward(const qmoe_gated_ffn_config* cfg, int64_t T, const void* dy, const void* x,
                                    const void* w1, const void* w2, const float* gu, void* dx, void* dw1, void* db1,
                                    void* dw2, void* db2, void* workspace, size_t workspace_bytes, void* stream) {
    GateParams gate;
    if (qmoe_status s = check_ffn(cfg, T, &gate)) return s;
    const int64_t H = cfg->hidden_size, I = cfg->inter_size;
    cudaStream_t st = (cudaStream_t)stream;
    if (misaligned(dx, 16) || misaligned(dw1, 16) || misaligned(dw2, 16) || misaligned(db1, 2) || misaligned(db2, 2))
        return bad(QMOE_INVALID_ARGUMENT, "gradients must be 16-byte, bias gradients 2-byte aligned");
    void* outs[] = {T ? dx : nullptr, dw1, db1, dw2, db2};
    const size_t bytes[] = {0, size_t(4 * I) * H, size_t(4 * I), size_t(2 * I) * H, size_t(2 * H)};
    void* first = nullptr;
    for (void* o : outs)
        if (o && !first) first = o;
    if (!first) return QMOE_OK;
    if (T == 0) {  // empty sums
        if (qmoe_status s = on_current_device(first)) return s;
        for (int i = 1; i < 5; ++i)
            if (outs[i])
                if (cudaError_t e = cudaMemsetAsync(outs[i], 0, bytes[i], st)) return cuda_bad(e, "gated_ffn_backward");
        return QMOE_OK;
    }
    if (!dy || !x || !w1 || !w2 || !gu) return bad(QMOE_INVALID_ARGUMENT, "dy, x, w1, w2 and gu are required");
    if (misaligned(dy, 16) || misaligned(x, 16) || misaligned(w1, 16) || misaligned(w2, 16) || misaligned(gu, 16))
        return bad(QMOE_INVALID_ARGUMENT, "tensors must be 16-byte aligned");
    const FfnLayout l(*cfg, T, true);
    if (qmoe_status s = check_workspace(workspace, workspace_bytes, l.total)) return s;
    if (qmoe_status s = on_current_device(first)) return s;
    char* ws = (char*)workspace;
    void *h = ws + l.h, *dgu = ws + l.dgu;
    float *sums = (float*)(ws + l.sums), *part = (float*)(ws + l.part);
    int64_t sum_rows = 0;
    cudaError_t e = cudaSuccess;
    auto product = [&](DenseOperand oa, DenseOperand ob, int64_t M, int64_t N, int64_t K, void* out) {
        DenseArgs a{};
        a.a = oa;
        a.b = ob;
        a.M = M;
        a.N = N;
        a.K = K;
        a.epi = kEpiStore;
        a.out = out;
        a.status = (int32_t*)workspace;
        return a;
    };
    if (dx || dw1 || db1 || dw2) {
        DenseArgs a{};
        a.a = rows_of(dy, H);
        a.b = cols_of(w2, I);
        a.M = T;
        a.N = I;
        a.K = H;
        a.epi = kEpiGateBwd;
        a.out = h;
        a.gu = const_cast<float*>(gu);
        a.dgu = dgu;
        a.sums = db1 ? sums : nullptr;
        a.gate = gate;
        a.interleaved = cfg->swiglu_fusion == 1;
        a.status = (int32_t*)workspace;
        a.reset_status = 1;
        sum_rows = dense_sum_rows(a);
        e = launch_rows(a, false, st);
    } else if (e == cudaSuccess) {
        e = cudaMemsetAsync(workspace, 0, 4, st);
    }
    const DenseArgs pdx = product(rows_of(dgu, 2 * I), cols_of(w1, H), T, H, 2 * I, dx);
    const DenseArgs pw1 = product(cols_of(dgu, 2 * I), cols_of(x, H), 2 * I, H, T, dw1);
    const DenseArgs pw2 = product(cols_of(dy, H), cols_of(h, I), H, I, T, dw2);
    const bool stream_dx = dx && dense_streams(T, 4 * I * H);
    if (e == cudaSuccess && stream_dx) e = launch_dense_stream(pdx, true, st);
    // h comes from the kernel before dx: known to be complete after dx's launch only
    if (e == cudaSuccess && ((dx && !stream_dx) || dw1 || dw2))
        e = launch_dense_pairs(dx && !stream_dx ? &pdx : nullptr, dw1 ? &pw1 : nullptr, dw2 ? &pw2 : nullptr, stream_dx,
                               st);
    if (e == cudaSuccess) e = launch_colsum({sums, sum_rows, 2 * I, db1}, {dy, T, H, db2}, part, st);
    return e == cudaSuccess ? QMOE_OK : cuda_bad(e, "gated_ffn_backward");
}

}  // extern "C"
