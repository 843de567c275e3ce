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
#include "dense.cuh"

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
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[i]));
        const __nv_bfloat162 q = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        const uint32_t m = *reinterpret_cast<const uint32_t*>(&q);
        return max(m << 16, m & 0xFFFF0000u);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, v[i] & 0x7FFFFFFFu);
    return m;
}

// The chunk of a warp: its row, the lane's first element in it and what is left
// of the row from there. One long row (every contiguous matrix) needs no
// division.
template <int EV>
__device__ __forceinline__ bool chunk_of(int64_t w, int64_t rows, int64_t K, int64_t& row, int64_t& k0, int& left) {
    constexpr int64_t WE = 32 * EV * kVec;
    const int64_t per_row = (K + WE - 1) / WE;
    if (w >= rows * per_row) return false;
    row = rows == 1 ? 0 : w / per_row;
    k0 = (w - row * per_row) * WE + (threadIdx.x & 31) * EV;
    left = int(min(K - k0, WE));
    return true;
}

// Code words and scale byte of a lane's vector.
template <bool BF16>
__device__ __forceinline__ uint32_t quantize_vector(const uint4& v, uint32_t& byte) {
    constexpr int LB = BF16 ? 4 : 8;  // lanes of a block
    uint32_t m = absmax_bits<BF16>(v);
#pragma unroll
    for (int o = 1; o < LB; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t r[4] = {v.x, v.y, v.z, v.w};
    const bool bad = m >= 0x7F800000u;
    byte = bad ? 255u : uint32_t(max(int(m >> 23) - 2, 0));
    uint32_t c;
    if (BF16) {
        // 2^(127 - byte) in both halves (anything for a bad block)
        const uint32_t inv = ((254u - byte) << 7) * 0x00010001u;
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // exact: a power of two, no overflow; what underflows has code 0
            const __nv_bfloat162 q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r[i]),
                                             *reinterpret_cast<const __nv_bfloat162*>(&inv));
            const uint32_t w = *reinterpret_cast<const uint32_t*>(&q);
            f[2 * i] = __uint_as_float(w << 16);
            f[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
        c = e2m1x8(f);
    } else {
        const float inv = __uint_as_float((254u - byte) << 23);
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(r[i]) * inv;
        c = e2m1x4(f);
    }
    return bad ? 0u : c;
}

__device__ __forceinline__ void tile_scales(const ScaleTiles& t, int64_t pitch, int64_t i, int64_t step) {
    const int subs = t.subs(), groups = (t.chunks + 3) / 4;  // 16 scales of a row
    const int64_t total = t.threads();
    for (; i < total; i += step) {
        const int64_t pr = i / groups;  // padded row
        const int g = int(i - pr * groups);
        const int64_t tile = pr / (subs * 128);
        const int r = int(pr - tile * subs * 128);
        const int64_t row = tile * t.tile_rows + r;
        uint32_t w[4] = {0, 0, 0, 0};
        if (r < t.tile_rows && row < t.rows) load_scales<4>(t.s, t.rows * pitch, row, pitch, g * 16, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = g * 4 + j;
            if (c < t.chunks)
                reinterpret_cast<uint32_t*>(t.out)[((tile * t.chunks + c) * subs + (r >> 7)) * 128 + (r & 31) * 4 +
                                                   ((r >> 5) & 3)] = w[j];
        }
    }
}

__global__ void __launch_bounds__(kThreads) mx4_tile_scales_kernel(const ScaleTiles a, const ScaleTiles b, int64_t pitch) {
    pdl_wait();
    pdl_trigger();
    tile_scales(blockIdx.y == 0 ? a : b, pitch, int64_t(blockIdx.x) * kThreads + threadIdx.x,
                int64_t(gridDim.x) * kThreads);
}

// TILED: the scales go to the order of the product's copies instead of rows,
// and the CTAs from `own` on lay out the other operand's scales (the work of
// one more launch).
template <bool BF16, bool TILED>
__global__ void __launch_bounds__(kThreads, 6) mx4_quantize_kernel(const uint8_t* x, int64_t rows, int64_t K, int64_t ldb,
                                                                   uint8_t* codes, uint8_t* scales, int own,
                                                                   const ScaleTiles to, const ScaleTiles other) {
    pdl_wait();
    pdl_trigger();
    if (TILED && int(blockIdx.x) >= own) {
        tile_scales(other, K / 32, int64_t(blockIdx.x - own) * kThreads + threadIdx.x,
                    int64_t(gridDim.x - own) * kThreads);
        return;
    }
    constexpr int EV = BF16 ? 8 : 4, ES = 16 / EV, STEP = 32 * EV;  // elements of a vector, bytes, elements of a warp's
    const int64_t nw = int64_t(own) * (kThreads / 32);
    const int64_t KW = TILED ? int64_t(to.chunks) * 128 : K;  // tiled scales end on a stage: zeros after K
    int64_t row, k0;
    int left;
    for (int64_t w = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); chunk_of<EV>(w, rows, KW, row, k0, left);
         w += nw) {
        const uint8_t* src = x + row * ldb + k0 * ES;
        const int have = TILED ? int(min(K - k0, int64_t(left))) : left;
        uint4 v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            v[j] = j * STEP < have ? __ldcs(reinterpret_cast<const uint4*>(src + j * STEP * ES)) : make_uint4(0, 0, 0, 0);
        const int64_t at = row * K + k0;
        uint8_t *cd = codes + at / 2, *sd = scales + at / 32;
        const bool first = (threadIdx.x & (32 / EV - 1)) == 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            uint32_t byte;
            const uint32_t c = quantize_vector<BF16>(v[j], byte);
            if (j * STEP < have) {
                if (BF16) *reinterpret_cast<uint32_t*>(cd + j * STEP / 2) = c;
                else *reinterpret_cast<uint16_t*>(cd + j * STEP / 2) = uint16_t(c);
            }
            if (first && j * STEP < left) {
                if (TILED) to.out[to.place(row, (k0 + j * STEP) / 32)] = uint8_t(byte);
                else sd[j * STEP / 32] = uint8_t(byte);
            }
        }
    }
}

// 2^(byte - 127) as bf16 bits; byte 0 is the subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ uint32_t e8m0_bf16(uint32_t byte) {
    return byte == 0 ? 0x0040u : byte == 255 ? 0x7FC0u : byte << 7;
}

// Four codes (the low 16 bits) to bf16 in order. The values' high and low
// bytes come from two eight-entry byte tables, four at a time (a byte
// permute's selectors are the codes' three magnitude bits); the sign comes
// from the permute's sign mode: of a table of 0x80, a selector with its fourth
// bit set gives 0xFF and any other 0x80, so bit 0 is the code's sign.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
__device__ __forceinline__ void e2m1x4_to_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t mag = c & 0x7777u;
    const uint32_t sign = (prmt(0x80808080u, 0x80808080u, c) & 0x01010101u) << 7;
    const uint32_t hb = prmt(0x3F3F3F00u, 0x40404040u, mag) | sign;
    const uint32_t lb = prmt(0xC0800000u, 0xC0804000u, mag);
    lo = __byte_perm(lb, hb, 0x5140);
    hi = __byte_perm(lb, hb, 0x7362);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                  int64_t rows, int64_t K, uint8_t* x, int64_t ldb) {
    pdl_wait();
    pdl_trigger();
    constexpr int EV = BF16 ? 8 : 4, ES = 16 / EV, STEP = 32 * EV;
    const int64_t nw = int64_t(gridDim.x) * (kThreads / 32);
    int64_t row, k0;
    int left;
    for (int64_t w = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); chunk_of<EV>(w, rows, K, row, k0, left);
         w += nw) {
        const int64_t at = row * K + k0;
        const uint8_t *cs = codes + at / 2, *ss = scales + at / 32;
        uint8_t* dst = x + row * ldb + k0 * ES;
        uint32_t c[kVec], s[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            c[j] = s[j] = 0;
            if (j * STEP < left) {
                c[j] = BF16 ? *reinterpret_cast<const uint32_t*>(cs + j * STEP / 2)
                            : *reinterpret_cast<const uint16_t*>(cs + j * STEP / 2);
                s[j] = ss[j * STEP / 32];
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (j * STEP >= left) break;
            // a code's value has two significant bits: its product with a power
            // of two is exact in bf16, subnormals included
            uint32_t o[4];
            const uint32_t sc = e8m0_bf16(s[j]) * 0x00010001u;
            if (BF16) {
                e2m1x4_to_bf16(c[j], o[0], o[1]);
                e2m1x4_to_bf16(c[j] >> 16, o[2], o[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&o[i]),
                                                     *reinterpret_cast<const __nv_bfloat162*>(&sc));
                    o[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
            } else {
                const float f = __uint_as_float(sc & 0xFFFF0000u);
                uint32_t v[2];
                e2m1x4_to_bf16(c[j], v[0], v[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    o[2 * i] = __float_as_uint(__uint_as_float(v[i] << 16) * f);
                    o[2 * i + 1] = __float_as_uint(__uint_as_float(v[i] & 0xFFFF0000u) * f);
                }
            }
            __stcs(reinterpret_cast<uint4*>(dst + j * STEP * ES), make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

int64_t round_grid(int64_t rows, int64_t K, int ev) {
    const int64_t we = 32 * ev * kVec;
    const int64_t ctas = (rows * ((K + we - 1) / we) + kThreads / 32 - 1) / (kThreads / 32);
    return ctas < (1 << 24) ? ctas : (1 << 24);
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                uint8_t* scales, cudaStream_t st) {
    const int64_t ldb = ldx * (bf16 ? 2 : 4);
    if (ldx == K) { K *= rows; rows = 1; }
    const int grid = int(round_grid(rows, K, bf16 ? 8 : 4));
    return launch_kernel(bf16 ? mx4_quantize_kernel<true, false> : mx4_quantize_kernel<false, false>, dim3(unsigned(grid)),
                         dim3(kThreads), 0, st, true, (const uint8_t*)x, rows, K, ldb, codes, scales, grid, ScaleTiles{},
                         ScaleTiles{});
}

cudaError_t launch_mx4_quantize_tiled(const void* x, int bf16, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                                      const ScaleTiles& to, const ScaleTiles& other, cudaStream_t st) {
    const int grid = int(round_grid(rows, int64_t(to.chunks) * 128, bf16 ? 8 : 4));
    const int64_t blocks = (other.threads() + kThreads - 1) / kThreads;
    const int more = int(blocks < 4096 ? blocks : 4096);
    return launch_kernel(bf16 ? mx4_quantize_kernel<true, true> : mx4_quantize_kernel<false, true>,
                         dim3(unsigned(grid + more)), dim3(kThreads), 0, st, true, (const uint8_t*)x, rows, K,
                         ldx * (bf16 ? 2 : 4), codes, (uint8_t*)nullptr, grid, to, other);
}

cudaError_t launch_mx4_tile_scales(const ScaleTiles& a, const ScaleTiles& b, int64_t K, cudaStream_t st) {
    const int64_t t = a.threads() > b.threads() ? a.threads() : b.threads(), blocks = (t + kThreads - 1) / kThreads;
    return launch_kernel(mx4_tile_scales_kernel, dim3(unsigned(blocks < 4096 ? blocks : 4096), 2), dim3(kThreads), 0, st,
                         true, a, b, K / 32);
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
