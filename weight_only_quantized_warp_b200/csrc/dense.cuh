// dense.cuh -- declarations shared by the dense operators' translation units:
// the gated activation with its derivatives, and the launchers of the MX4
// rounding kernels and of the products.
#pragma once

#include "qmoe_internal.cuh"

namespace qmoe {

// Gated activation of one (gate, up) pair. act: QMOE_ACT_* or kActGeluTanh;
// limit is +inf where nothing is clamped.
struct GateParams {
    int act;
    float alpha, beta, limit;
};

// A clamp that lets NaN through (both comparisons fail).
__device__ __forceinline__ float clamp_hi(float v, float hi) { return v > hi ? hi : v; }
__device__ __forceinline__ float clamp_lo(float v, float lo) { return v < lo ? lo : v; }

// Value and slope of the activation at g (slope skipped when not asked for).
// Fast exponentials and division: about 2^-21 relative, far inside the bf16
// rounding that every result goes through.
template <bool SLOPE>
__device__ __forceinline__ float gate_act(const GateParams& p, float g, float& slope) {
    switch (p.act) {
        case QMOE_ACT_RELU:
            if (SLOPE) slope = g > 0.0f ? 1.0f : (g <= 0.0f ? 0.0f : g);
            return g < 0.0f ? 0.0f : g;
        case QMOE_ACT_GELU: {
            const float cdf = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
            if (SLOPE) slope = cdf + g * 0.39894228040143268f * __expf(-0.5f * g * g);
            return g * cdf;
        }
        case kActGeluTanh: {
            const float c = 0.79788456080286536f, t = tanhf(c * (g + 0.044715f * g * g * g));
            if (SLOPE) slope = 0.5f * (1.0f + t) + 0.5f * g * (1.0f - t * t) * c * (1.0f + 0.134145f * g * g);
            return 0.5f * g * (1.0f + t);
        }
        case QMOE_ACT_SILU:
        case QMOE_ACT_SWIGLU: {
            const float a = p.act == QMOE_ACT_SILU ? 1.0f : p.alpha;
            const float s = __fdividef(1.0f, 1.0f + __expf(-a * g));
            if (SLOPE) slope = s + a * g * s * (1.0f - s);
            return g * s;
        }
        default:
            if (SLOPE) slope = 1.0f;
            return g;
    }
}

// h = act(g') (u' + beta), with SwiGLU's clamps g' and u'.
__device__ __forceinline__ float gate_value(const GateParams& p, float g, float u) {
    float none;
    if (p.act == QMOE_ACT_SWIGLU) {
        g = clamp_hi(g, p.limit);
        u = clamp_lo(clamp_hi(u, p.limit), -p.limit) + p.beta;
    }
    return gate_act<false>(p, g, none) * u;
}

// h and its derivatives by the unclamped g and u.
__device__ __forceinline__ float gate_slopes(const GateParams& p, float g, float u, float& hg, float& hu) {
    float gin = 1.0f, uin = 1.0f;
    if (p.act == QMOE_ACT_SWIGLU) {
        gin = g > p.limit ? 0.0f : 1.0f;
        uin = u > p.limit || u < -p.limit ? 0.0f : 1.0f;
        g = clamp_hi(g, p.limit);
        u = clamp_lo(clamp_hi(u, p.limit), -p.limit) + p.beta;
    }
    float slope;
    const float a = gate_act<true>(p, g, slope);
    hg = gin * slope * u;
    hu = uin * a;
    return a * u;
}

// ----------------------------------------------------------------- launchers
cudaError_t launch_mx4_quantize(const void* x, int bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                uint8_t* scales, cudaStream_t st);
cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* x,
                                  int bf16, int64_t ldx, cudaStream_t st);

// One operand of a product: element (r, k) at p + r * row + k * k_step (bf16
// elements), or MX4 rows (codes p, scales s).
struct DenseOperand {
    const void* p;
    const uint8_t* s;
    int64_t row, k_step;
};

enum DenseEpilogue : int {
    kEpiStore = 0,   // out[m, n] = acc + bias[n]
    kEpiGate = 1,    // B rows are (gate, up) pairs: out = h [M, N/2], gu kept when not null
    kEpiGateBwd = 2  // acc = dh [M, N]; from gu: dgu [M, 2N] and h [M, N]
};

// D[m, n] = sum_k A(m, k) B(n, k), m < M, n < N, and its epilogue.
struct DenseArgs {
    DenseOperand a, b;
    int64_t M, N, K;
    int mx4;
    int epi;
    int out_f32;           // kEpiStore: fp32 output and bias, otherwise bf16
    const void* bias;      // kEpiStore: [N]; kEpiGate: [N] bf16 in w1's row order; nullable
    void* out;             // kEpiStore: [M, N]; kEpiGate, kEpiGateBwd: h
    float* gu;             // kEpiGate: written when not null; kEpiGateBwd: read
    void* dgu;             // kEpiGateBwd
    GateParams gate;
    int interleaved;       // gate and up interleaved in w1 / gu (else concatenated)
    int32_t* status;       // workspace status word; reset by the call's first product
    int reset_status;
    void* scratch;         // mx4: dense_pair_workspace bytes
};
size_t dense_pair_workspace(int64_t M, int64_t N, int64_t K);  // re-laid MX4 scales
cudaError_t launch_dense_pair(const DenseArgs& a, cudaStream_t st);

// The same for few rows of A (kEpiStore and kEpiGate, both operands along k):
// M up to kStreamRows. `after` says that the kernel before it on the stream,
// which wrote A, may still be running (it triggers programmatic launch).
constexpr int64_t kStreamRows = 64;
cudaError_t launch_dense_stream(const DenseArgs& a, bool after, cudaStream_t st);

// out[n] = sum_m x[m, n] (x [M, N] bf16) in a fixed order; part: workspace of
// colsum_bytes(M, N).
size_t colsum_bytes(int64_t M, int64_t N);
cudaError_t launch_colsum(const void* x, int64_t M, int64_t N, void* out, float* part, cudaStream_t st);

}  // namespace qmoe
