// dense.cuh -- declarations shared by the dense operators' translation units:
// the gated activation with its derivatives, and the launchers of the MX4
// rounding kernels and of the products.
#pragma once

#include "qmoe_internal.cuh"

namespace qmoe {

// Gated activation of one (gate, up) pair, h = act(g') (u' + beta) with
// g' = min(g, limit) and u' = clamp(u, -limit, limit) (limit is +inf and beta 0
// except for SwiGLU). act(g) = g s(g), where s is
//   kGateSigmoid   1 / (1 + exp(-z)), z = g (c1 + c3 g^2): SiLU and SwiGLU with
//                  c3 = 0, and tanh-form GELU, since (1 + tanh v) / 2 is the
//                  sigmoid of 2 v
//   kGateErf       the normal distribution function
//   kGateStep      1 for g > 0, else 0 (ReLU)
//   kGateOne       1
// so that one short piece of code, unrolled over a thread's elements, serves
// every activation (six inlined bodies overflowed the instruction cache: the
// gradient epilogue then took 60 us for one tile's rows, all of it fetching).
enum : int { kGateSigmoid = 0, kGateErf = 1, kGateStep = 2, kGateOne = 3 };
struct GateParams {
    int mode;
    float c1, c3, beta, limit;
};

// Clamps that let NaN through (both comparisons fail).
__device__ __forceinline__ float clamp_hi(float v, float hi) { return v > hi ? hi : v; }
__device__ __forceinline__ float clamp_lo(float v, float lo) { return v < lo ? lo : v; }

// act(g), and its slope when asked for: s + g s'(g). Fast exponentials and
// division: about 2^-21 relative, far inside the bf16 rounding that every
// result goes through.
template <bool SLOPE>
__device__ __forceinline__ float gate_act(const GateParams& p, float g, float& slope) {
    if (p.mode == kGateSigmoid) {
        const float g2 = g * g, s = __fdividef(1.0f, 1.0f + __expf(-g * fmaf(p.c3, g2, p.c1)));
        if (SLOPE) slope = fmaf(g * fmaf(3.0f * p.c3, g2, p.c1), s * (1.0f - s), s);
        return g * s;
    }
    if (p.mode == kGateErf) {
        const float s = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
        if (SLOPE) slope = fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), s);
        return g * s;
    }
    const bool on = p.mode == kGateOne || g > 0.0f;
    if (SLOPE) slope = on ? 1.0f : (g <= 0.0f ? 0.0f : g);
    return on || !(g <= 0.0f) ? g : 0.0f;
}

__device__ __forceinline__ float gate_value(const GateParams& p, float g, float u) {
    float none;
    return gate_act<false>(p, clamp_hi(g, p.limit), none) * (clamp_lo(clamp_hi(u, p.limit), -p.limit) + p.beta);
}

// h and its derivatives by g and u (0 beyond a clamp).
__device__ __forceinline__ float gate_slopes(const GateParams& p, float g, float u, float& hg, float& hu) {
    float slope;
    const float a = gate_act<true>(p, clamp_hi(g, p.limit), slope);
    const float f = clamp_lo(clamp_hi(u, p.limit), -p.limit) + p.beta;
    hg = g > p.limit ? 0.0f : slope * f;
    hu = fabsf(u) > p.limit ? 0.0f : a;
    return a * f;
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

// The same for few rows of A (along k): M up to kStreamRows. early_w: B was not
// written by the kernel before this one on the stream, so loads of it need not
// wait for that kernel.
constexpr int64_t kStreamRows = 64;
cudaError_t launch_dense_stream(const DenseArgs& a, bool early_w, cudaStream_t st);

// out[n] = sum_m x[m, n] (x [M, N] bf16) in a fixed order; part: workspace of
// colsum_bytes(M, N).
size_t colsum_bytes(int64_t M, int64_t N);
cudaError_t launch_colsum(const void* x, int64_t M, int64_t N, void* out, float* part, cudaStream_t st);

}  // namespace qmoe
