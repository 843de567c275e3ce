// dense_colsum.cu -- column sums of one or two matrices (the bias gradients: of
// the gate-backward launch's fp32 sums of 32 tokens each, and of dy in bf16),
// sm_100a. HBM-bound: one read of the matrices. The rows are cut into S ranges; a
// CTA sums 256 columns of one range (eight warps take alternate rows, a lane 16
// or 32 bytes, joined through shared memory in warp order) and a second kernel
// adds the S partials in order, so the result does not depend on timing. Both
// matrices share the launches: at T = 1023 and 5760 + 2880 columns four launches
// took 22 us, two take 11.
#include "dense.cuh"

namespace qmoe {
namespace {

constexpr int kColWarps = 8;

// Columns of both matrices side by side, 256 a CTA: a's first.
struct ColPair {
    ColSum a, b;            // fp32, bf16
    int blocks_a;
    int ranges_a, ranges_b;  // of their rows
};

__device__ __forceinline__ bool col_block(const ColPair& p, int64_t& c0) {
    const bool second = int(blockIdx.x) >= p.blocks_a;
    c0 = int64_t(int(blockIdx.x) - (second ? p.blocks_a : 0)) * 256;
    return second;
}

__global__ void __launch_bounds__(kColWarps * 32) colsum_part_kernel(const ColPair p, float* part) {
    __shared__ float sum[kColWarps][256];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t c0;
    const bool bf16 = col_block(p, c0);
    const ColSum& s = bf16 ? p.b : p.a;
    const int ranges = bf16 ? p.ranges_b : p.ranges_a;
    if (int(blockIdx.y) >= ranges) return;
    const int64_t per = (s.M + ranges - 1) / ranges;
    const int64_t c = c0 + lane * 8;  // N is a multiple of 8
    const int64_t m0 = blockIdx.y * per, m1 = min(s.M, m0 + per);
    float acc[8] = {};
    if (c < s.N && bf16) {
        const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(s.x);
#pragma unroll 4
        for (int64_t m = m0 + warp; m < m1; m += kColWarps) {
            const uint4 v = *reinterpret_cast<const uint4*>(x + m * s.N + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] += __uint_as_float(w[i] << 16);
                acc[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    } else if (c < s.N) {
        const float* x = reinterpret_cast<const float*>(s.x);
#pragma unroll 4
        for (int64_t m = m0 + warp; m < m1; m += kColWarps) {
            const float4 v = *reinterpret_cast<const float4*>(x + m * s.N + c);
            const float4 w = *reinterpret_cast<const float4*>(x + m * s.N + c + 4);
            acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
            acc[4] += w.x; acc[5] += w.y; acc[6] += w.z; acc[7] += w.w;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[warp][lane * 8 + i] = acc[i];
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kColWarps; ++w) t += sum[w][threadIdx.x];
    part[(int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x] = t;
}

__global__ void __launch_bounds__(256) colsum_join_kernel(const ColPair p, const float* part) {
    pdl_wait();
    pdl_trigger();
    int64_t c0;
    const bool bf16 = col_block(p, c0);
    const ColSum& s = bf16 ? p.b : p.a;
    const int ranges = bf16 ? p.ranges_b : p.ranges_a;
    const int64_t c = c0 + threadIdx.x;
    if (c >= s.N) return;
    float t = 0.0f;
#pragma unroll 8
    for (int i = 0; i < ranges; ++i) t += part[(int64_t(i) * gridDim.x + blockIdx.x) * 256 + threadIdx.x];
    reinterpret_cast<__nv_bfloat16*>(s.out)[c] = __float2bfloat16_rn(t);
}

int64_t col_blocks(int64_t N) { return (N + 255) / 256; }

// Row ranges of a matrix: about four CTAs for each SM of a B200 (the size of a
// workspace follows from them and is asked for without a device), at least 32
// rows each. They are those of both sums whichever is asked for, so that either
// comes out the same alone.
int col_ranges(int64_t M, int64_t Na, int64_t Nb) {
    const int64_t blocks = col_blocks(Na) + col_blocks(Nb);
    const int64_t want = (4 * 148 + blocks - 1) / blocks, most = (M + 31) / 32;
    return int(want < most ? want : most);
}

}  // namespace

size_t colsum_bytes(int64_t Ma, int64_t Na, int64_t Mb, int64_t Nb) {
    return size_t((col_blocks(Na) + col_blocks(Nb)) * col_ranges(Ma > Mb ? Ma : Mb, Na, Nb)) * 1024;
}

cudaError_t launch_colsum(const ColSum& a, const ColSum& b, float* part, cudaStream_t st) {
    const int64_t blocks_a = a.out ? col_blocks(a.N) : 0, blocks = blocks_a + (b.out ? col_blocks(b.N) : 0);
    if (blocks == 0) return cudaSuccess;
    const ColPair p{a, b, int(blocks_a), col_ranges(a.M, a.N, b.N), col_ranges(b.M, a.N, b.N)};
    const int ya = a.out ? p.ranges_a : 0, yb = b.out ? p.ranges_b : 0;
    const cudaError_t e = launch_kernel(colsum_part_kernel, dim3(unsigned(blocks), unsigned(ya > yb ? ya : yb)),
                                        dim3(kColWarps * 32), 0, st, true, p, part);
    if (e != cudaSuccess) return e;
    return launch_kernel(colsum_join_kernel, dim3(unsigned(blocks)), dim3(256), 0, st, true, p, (const float*)part);
}

}  // namespace qmoe
