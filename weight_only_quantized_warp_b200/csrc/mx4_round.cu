// mx4_round.cu -- rows to 4-bit microscaling blocks and back (sm_100a).
//
// A block is 32 consecutive k of one row. With m the block's largest
// magnitude, the shared scale is 2^E, E = floor(log2 m) - 2 (2 is the exponent
// of the largest e2m1 magnitude, 6), held as the byte E + 127 and clamped at
// 0; each element becomes the e2m1 code nearest to x / 2^E, ties to the even
// code, magnitudes above 6 (m in (6, 8) 2^E) to 6. The division is a product
// with the power of two 2^-E, which fp32 holds exactly for every E that
// occurs (127 .. -125), so codes are decided exactly. A block with a NaN or
// an infinity has no scale: its byte is 255 (NaN) and its codes are 0.
//
// Both directions are HBM-bound: (s + 17/32) bytes per element for elements
// of s bytes, about ten instructions. Each lane takes 16 bytes of x at a time
// (a block is 4 lanes of bf16 or 8 of fp32, joined by shuffles), kVec of them
// in flight; a row that continues in the next (ldx = K) is walked as one long
// row.
#include "qmoe_internal.cuh"

namespace qmoe {
namespace {

constexpr int kVec = 4;         // 16-byte vectors of x a lane holds at once
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ uint32_t e2m1x4(const float (&v)[4]) {
    uint32_t r;
    asm("{\n.reg .b8 a, b, z;\n.reg .b16 h;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "mov.b16 h, {a, b};\ncvt.u32.u16 %0, h;\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
    return r;
}

// Largest magnitude of the lane's vector as fp32 bits (a NaN's bits exceed
// every number's, so an integer maximum carries it).
template <bool BF16>
__device__ __forceinline__ uint32_t absmax_bits(const uint4& w) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    if (BF16) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
        return max(m << 16, m & 0xFFFF0000u);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, v[i] & 0x7FFFFFFFu);
    return m;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(const uint8_t* x, int64_t rows, int64_t K,
                                                                int64_t ldb, uint8_t* codes,
                                                                uint8_t* scales) {
    pdl_wait();
    pdl_trigger();
    constexpr int EV = BF16 ? 8 : 4;            // elements of a vector
    constexpr int LB = 32 / EV;                 // lanes of a block
    constexpr int64_t WE = 32 * EV * kVec;      // elements a warp takes at once
    const int lane = threadIdx.x & 31;
    const int64_t nw = int64_t(gridDim.x) * (kThreads / 32);
    const int64_t per_row = (K + WE - 1) / WE;
    for (int64_t w = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); w < rows * per_row; w += nw) {
        const int64_t row = w / per_row;
        const int64_t k0 = (w - row * per_row) * WE + lane * EV;
        const uint8_t* src = x + row * ldb;
        uint4 v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t k = k0 + j * 32 * EV;
            v[j] = k < K ? __ldcs(reinterpret_cast<const uint4*>(src + k * (16 / EV))) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t k = k0 + j * 32 * EV;
            uint32_t m = absmax_bits<BF16>(v[j]);
#pragma unroll
            for (int o = 1; o < LB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const bool bad = m >= 0x7F800000u;
            const int be = int(m >> 23);
            const uint32_t byte = bad ? 255u : uint32_t(max(be - 2, 0));
            const float inv = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte); unused when bad
            const uint32_t r[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            uint32_t c;
            if (BF16) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = __uint_as_float(r[i] << 16) * inv;
                    f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u) * inv;
                }
                c = e2m1x8(f);
            } else {
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]) * inv;
                c = e2m1x4(f);
            }
            if (bad) c = 0;
            if (k < K) {
                uint8_t* d = codes + (row * K + k) / 2;
                if (BF16) *reinterpret_cast<uint32_t*>(d) = c;
                else *reinterpret_cast<uint16_t*>(d) = uint16_t(c);
                if ((lane & (LB - 1)) == 0) scales[(row * K + k) / 32] = uint8_t(byte);
            }
        }
    }
}

// 2^(byte - 127); byte 0 is the fp32 subnormal 2^-127, byte 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// Magnitude by the code's low three bits, twice over: (1 + m/2) 2^(e-1).
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const float mag = e == 0 ? 0.5f * float(m) : __uint_as_float(((e + 126u) << 23) | (m << 22));
    return (c & 8u) ? -mag : mag;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint8_t* codes,
                                                                  const uint8_t* scales, int64_t rows,
                                                                  int64_t K, uint8_t* x, int64_t ldb) {
    pdl_wait();
    pdl_trigger();
    constexpr int EV = BF16 ? 8 : 4;
    constexpr int64_t WE = 32 * EV * kVec;
    const int lane = threadIdx.x & 31;
    const int64_t nw = int64_t(gridDim.x) * (kThreads / 32);
    const int64_t per_row = (K + WE - 1) / WE;
    for (int64_t w = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); w < rows * per_row; w += nw) {
        const int64_t row = w / per_row;
        const int64_t k0 = (w - row * per_row) * WE + lane * EV;
        uint32_t c[kVec], s[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t k = k0 + j * 32 * EV;
            c[j] = s[j] = 0;
            if (k < K) {
                const uint8_t* p = codes + (row * K + k) / 2;
                c[j] = BF16 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
                s[j] = scales[(row * K + k) / 32];
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t k = k0 + j * 32 * EV;
            if (k >= K) continue;
            const float sc = e8m0_value(s[j]);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BF16) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(e2m1_value(c[j] >> (8 * i)) * sc,
                                                                   e2m1_value(c[j] >> (8 * i + 4)) * sc);
                    o[i] = *reinterpret_cast<const uint32_t*>(&b);
                } else {
                    o[i] = __float_as_uint(e2m1_value(c[j] >> (4 * i)) * sc);
                }
            }
            __stcs(reinterpret_cast<uint4*>(x + row * ldb + k * (16 / EV)), make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

int64_t round_grid(int64_t rows, int64_t K, int ev) {
    const int64_t we = 32 * ev * kVec;
    const int64_t ctas = (rows * ((K + we - 1) / we) + kThreads / 32 - 1) / (kThreads / 32);
    return ctas < 148 * 16 ? ctas : 148 * 16;
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                uint8_t* scales, cudaStream_t st) {
    const int64_t ldb = ldx * (bf16 ? 2 : 4);
    if (ldx == K) { K *= rows; rows = 1; }
    const int grid = int(round_grid(rows, K, bf16 ? 8 : 4));
    return launch_kernel(bf16 ? mx4_quantize_kernel<true> : mx4_quantize_kernel<false>, dim3(unsigned(grid)),
                         dim3(kThreads), 0, st, true, (const uint8_t*)x, rows, K, ldb, codes, scales);
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, void* x,
                                  int bf16, int64_t ldx, cudaStream_t st) {
    const int64_t ldb = ldx * (bf16 ? 2 : 4);
    if (ldx == K) { K *= rows; rows = 1; }
    const int grid = int(round_grid(rows, K, bf16 ? 8 : 4));
    return launch_kernel(bf16 ? mx4_dequantize_kernel<true> : mx4_dequantize_kernel<false>, dim3(unsigned(grid)),
                         dim3(kThreads), 0, st, true, codes, scales, rows, K, (uint8_t*)x, ldb);
}

}  // namespace qmoe
