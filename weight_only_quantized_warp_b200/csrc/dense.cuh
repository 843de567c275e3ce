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
// The wide epilogues branch on s once per block of elements (with_gate_mode), so
// the code they run is short and straight: with the branch inside the unrolled
// element loop they were bound by instruction fetches (128 x 80 columns of h
// took 10 us against 5, one tile of the backward pass 60 us with all six
// activations inlined). The streaming kernel's few elements branch one by one:
// copies of its code for each s measured slower (a token's block 64 against 61
// us, a training step of 64 tokens 45 against 43).
enum : int { kGateSigmoid = 0, kGateErf = 1, kGateStep = 2, kGateOne = 3 };
struct GateParams {
    int mode;
    float c1, c3, beta, limit;
};

// Clamps that let NaN through (both comparisons fail).
__device__ __forceinline__ float clamp_hi(float v, float hi) { return v > hi ? hi : v; }
__device__ __forceinline__ float clamp_lo(float v, float lo) { return v < lo ? lo : v; }

template <int MODE>
__device__ __forceinline__ bool gate_is(const GateParams& p, int mode) {
    return MODE < 0 ? p.mode == mode : MODE == mode;
}

// act(g), and its slope when asked for: s + g s'(g). MODE is the mode, or -1 to
// branch here. Far inside the bf16 rounding (2^-9) that every result goes
// through, down to the smallest s: the sigmoid's fast exponential and division
// are off by less than 2^-14 relative where s is near 1e-38 and 2^-20 where |z|
// is small, the normal distribution function by less than 2^-15 at g = -12.
template <int MODE, bool SLOPE>
__device__ __forceinline__ float gate_act(const GateParams& p, float g, float& slope) {
    if (gate_is<MODE>(p, kGateSigmoid)) {
        const float g2 = fminf(g * g, 3e38f);  // finite, so that 0 times it is 0 (from |g| = 1.8e19 on)
        const float s = __fdividef(1.0f, 1.0f + __expf(-g * fmaf(p.c3, g2, p.c1)));
        if (SLOPE) {  // where s has reached 0 or 1, z' may have overflowed
            const float q = s * (1.0f - s);
            slope = q > 0.0f ? fmaf(g * fmaf(3.0f * p.c3, g2, p.c1), q, s) : s;
        }
        return g * s;
    }
    if (gate_is<MODE>(p, kGateErf)) {
        // The tail beyond |g| as exp(-g^2 / 2) t P(t), t = 1 / (1 + 0.36 |g|). What
        // is left of the tail without its exponential is smooth and falls like
        // 1 / |g|; P is a polynomial of degree 6 fitted to it over t for the
        // smallest relative error (2^-19.6 for |g| <= 14). The form (1 + erf) / 2
        // cancels instead (4 % off at g = -5).
        const float e = __expf(-0.5f * g * g), t = __fdividef(1.0f, fmaf(0.36f, fabsf(g), 1.0f));
        float r = fmaf(0.0470560938f, t, -0.179764032f);
        r = fmaf(r, t, 0.180953145f);
        r = fmaf(r, t, 0.0265498906f);
        r = fmaf(r, t, 0.139719069f);
        r = fmaf(r, t, 0.141772479f);
        r = fmaf(r, t, 0.143713042f) * t * e;
        const float s = g < 0.0f ? r : 1.0f - r;
        if (SLOPE) slope = fmaf(g * 0.39894228040143268f, e, s);
        return g * s;
    }
    const bool on = gate_is<MODE>(p, kGateOne) || g > 0.0f;
    if (SLOPE) slope = on ? 1.0f : (g <= 0.0f ? 0.0f : g);
    return on || !(g <= 0.0f) ? g : 0.0f;
}

// CLAMP false: the limit is +inf.
template <int MODE, bool CLAMP>
__device__ __forceinline__ float gate_value(const GateParams& p, float g, float u) {
    float none;
    if (CLAMP) {
        g = clamp_hi(g, p.limit);
        u = clamp_lo(clamp_hi(u, p.limit), -p.limit);
    }
    return gate_act<MODE, false>(p, g, none) * (u + p.beta);
}

// h and its derivatives by g and u (0 beyond a clamp).
template <int MODE, bool CLAMP>
__device__ __forceinline__ float gate_slopes(const GateParams& p, float g, float u, float& hg, float& hu) {
    float slope;
    const float a = gate_act<MODE, true>(p, CLAMP ? clamp_hi(g, p.limit) : g, slope);
    const float f = (CLAMP ? clamp_lo(clamp_hi(u, p.limit), -p.limit) : u) + p.beta;
    hg = CLAMP && g > p.limit ? 0.0f : slope * f;
    hu = CLAMP && fabsf(u) > p.limit ? 0.0f : a;
    return a * f;
}

// f(GateMode<mode of p, whether it clamps>()).
template <int MODE, bool CLAMP>
struct GateMode {
    static constexpr int value = MODE;
    static constexpr bool clamp = CLAMP;
};
template <typename F>
__device__ __forceinline__ void with_gate_mode(const GateParams& p, F&& f) {
    if (p.mode == kGateSigmoid) {
        if (p.limit < INFINITY) f(GateMode<kGateSigmoid, true>());
        else f(GateMode<kGateSigmoid, false>());
    } else if (p.mode == kGateErf) {
        f(GateMode<kGateErf, false>());
    } else if (p.mode == kGateStep) {
        f(GateMode<kGateStep, false>());
    } else {
        f(GateMode<kGateOne, false>());
    }
}

// 4 NW consecutive scales of a row of `pitch` scales, from scale k0 on (a
// multiple of 4), as words; 0 past the row's end. The array starts on 4 bytes
// and holds `total` of them; rows need not be aligned, so a row's words are
// joined from the aligned words that hold them.
template <int NW>
__device__ __forceinline__ void load_scales(const uint8_t* s, int64_t total, int64_t row, int64_t pitch, int64_t k0,
                                            uint32_t (&w)[NW]) {
    const int64_t at = row * pitch + k0;
    const int n = int(min(int64_t(4 * NW), max(int64_t(0), pitch - k0)));  // bytes of the row
    if (NW % 4 == 0 && ((pitch | reinterpret_cast<uintptr_t>(s)) & 15) == 0 && (k0 & 15) == 0) {
#pragma unroll
        for (int j = 0; j < NW / 4; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (16 * j < n) v = reinterpret_cast<const uint4*>(s + at)[j];
            w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
        }
        return;
    }
    const int sh = int(at & 3);
    const int64_t a0 = at - sh;
    uint32_t r[NW + 1];
#pragma unroll
    for (int j = 0; j <= NW; ++j) {
        const int64_t p = a0 + 4 * j;
        r[j] = 0;
        if (4 * j < n + sh) {
            if (p + 4 <= total) {
                r[j] = *reinterpret_cast<const uint32_t*>(s + p);
            } else {  // the array's last bytes
                for (int b = 0; b < 4; ++b)
                    if (p + b < total) r[j] |= uint32_t(s[p + b]) << (8 * b);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NW; ++j) {
        w[j] = __funnelshift_r(r[j], r[j + 1], 8 * sh);
        const int left = n - 4 * j;
        if (left < 4) w[j] &= left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    }
}

// MX4 scales [rows, K/32] in the order in which the CTA-pair product copies
// them: [tile of tile_rows rows][chunk of 128 k][ceil(tile_rows / 128)][32][4]
// words of four scales, the word of row r (in its tile) at lane r % 32, column
// r / 32 % 4. Rows and scales past the end are 0 (their codes are zero).
struct ScaleTiles {
    const uint8_t* s;  // by rows
    uint8_t* out;      // tiled
    int64_t rows;
    int tile_rows, tiles, chunks;
    __host__ __device__ int subs() const { return (tile_rows + 127) / 128; }
    __host__ __device__ int64_t threads() const { return int64_t(tiles) * subs() * 128 * ((chunks + 3) / 4); }
    __host__ __device__ int64_t bytes() const { return int64_t(tiles) * chunks * subs() * 512; }
    // the byte of a row's scale j; tile_rows is 128 here
    __device__ int64_t place(int64_t row, int64_t j) const {
        const int r = int(row & 127);
        return ((row >> 7) * chunks + (j >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (j & 3);
    }
};

// What the products' bounded device waits take from qmoe_dense_set_option, read
// when a product is launched.
struct DenseWaits {
    uint64_t limit_ns;
    int withhold;  // test only: the MMA warp keeps back its first accumulator's signal
};
DenseWaits dense_waits();

// A count on the current device that goes up whenever a wait of the kernel gives
// up; read when the work before on the stream is done.
cudaError_t dense_pair_gave_up(uint32_t* count, cudaStream_t st);
cudaError_t dense_stream_gave_up(uint32_t* count, cudaStream_t st);

// ----------------------------------------------------------------- launchers
cudaError_t launch_mx4_quantize(const void* x, int bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                uint8_t* scales, cudaStream_t st);
cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* x,
                                  int bf16, int64_t ldx, cudaStream_t st);

// Quantise rows of x with their scales tiled (`to`; rows past the end are left
// as they are: a row's scales enter its own results only), and tile the scales
// of the product's other operand, in one launch; or tile both operands' scales.
cudaError_t launch_mx4_quantize_tiled(const void* x, int bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                      const ScaleTiles& to, const ScaleTiles& other, cudaStream_t st);
cudaError_t launch_mx4_tile_scales(const ScaleTiles& a, const ScaleTiles& b, int64_t K, cudaStream_t st);

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
    float* sums;           // kEpiGateBwd: [dense_sum_rows, 2N], sums over tokens of the unrounded dgu; nullable
    GateParams gate;
    int interleaved;       // gate and up interleaved in w1 / gu (else concatenated)
    int32_t* status;       // workspace status word; reset by the call's first product
    int reset_status;
    void* scratch;         // mx4: dense_pair_workspace bytes, holding both operands' tiled scales
};
// The tiled scales of an MX4 product's operands (their `s` left out) in a
// scratch of dense_pair_workspace(M, N, K) bytes.
void dense_pair_tiles(int64_t M, int64_t N, int64_t K, void* scratch, ScaleTiles* a, ScaleTiles* b);
size_t dense_pair_workspace(int64_t M, int64_t N, int64_t K);
// early: B was not written by the kernel before this one on the stream, so loads
// of it need not wait for that kernel.
cudaError_t launch_dense_pair(const DenseArgs& a, bool early, cudaStream_t st);

// Up to three plain products (kEpiStore, bf16, B across its rows) in one launch,
// any of them null: a long one, and two of the same K that fill in around it.
// B of the first two was not written by the kernel before this one; early3 says
// so of the third.
cudaError_t launch_dense_pairs(const DenseArgs* first, const DenseArgs* second, const DenseArgs* third, bool early3,
                               cudaStream_t st);

// The same for few rows of A (along k), streaming B: M up to 128. It is taken up
// to 64 rows, and up to 128 where B is so large (32 MB) that reading it outlasts
// the joining of more rows' partials. Measured, streaming against CTA pairs: the
// block H = 4096, I = 14336 71 against 100 us at 64 rows and 83 against 102 at
// 128, its dh and dx 73 against 137 and 102 against 138; H = 2048, I = 1408 17
// against 19.5 us at 64 rows, 27 against 20 at 128; MX4 of 14336 x 4096 and 64
// rows 14.9 against 15.2, of 2880 x 2880 10.5 against 8.9.
inline bool dense_streams(int64_t M, int64_t b_bytes) {
    return M <= 64 || (M <= 128 && b_bytes >= (int64_t(32) << 20));
}
cudaError_t launch_dense_stream(const DenseArgs& a, bool early, cudaStream_t st);

// Rows of DenseArgs::sums that a product of few rows or of many writes (one for
// each split of K, which finishes some of the tokens, or for 32 tokens), and the
// most that it may be.
int64_t dense_stream_splits(const DenseArgs& a);
inline int64_t dense_sum_rows(const DenseArgs& a) {
    return dense_streams(a.M, a.N * a.K * 2) ? dense_stream_splits(a) : (a.M + 31) / 32;
}
inline int64_t dense_sum_rows_most(int64_t M, int64_t N, int64_t K) {
    return dense_streams(M, N * K * 2) ? 8 : (M + 31) / 32;
}

// out[n] = sum_m x[m, n] (x [M, N] fp32 or bf16, out bf16; skipped when out is
// null) in a fixed order, for up to two matrices: an fp32 and a bf16 one; part:
// workspace of colsum_bytes.
struct ColSum {
    const void* x;
    int64_t M, N;
    void* out;
};
size_t colsum_bytes(int64_t Ma, int64_t Na, int64_t Mb, int64_t Nb);
cudaError_t launch_colsum(const ColSum& f32, const ColSum& bf16, float* part, cudaStream_t st);

}  // namespace qmoe
