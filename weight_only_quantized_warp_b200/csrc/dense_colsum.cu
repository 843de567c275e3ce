// dense_colsum.cu -- column sums of a bf16 matrix (the bias gradients),
// sm_100a. HBM-bound: one read of the matrix. The rows are cut into S ranges;
// a CTA sums 256 columns of one range (eight warps take alternate rows, a lane
// 16 bytes, joined through shared memory in warp order) and a second kernel
// adds the S partials in order, so the result does not depend on timing.
#include "dense.cuh"

namespace qmoe {
namespace {

constexpr int kColWarps = 8;

__global__ void __launch_bounds__(kColWarps * 32) colsum_part_kernel(const __nv_bfloat16* x, int64_t M,
                                                                    int64_t N, int64_t rows_per,
                                                                    float* part) {
    __shared__ float sum[kColWarps][256];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = int64_t(blockIdx.x) * 256 + lane * 8;  // N is a multiple of 8
    const int64_t m0 = blockIdx.y * rows_per, m1 = min(M, m0 + rows_per);
    float acc[8] = {};
    if (c < N) {
#pragma unroll 4
        for (int64_t m = m0 + warp; m < m1; m += kColWarps) {
            const uint4 v = *reinterpret_cast<const uint4*>(x + m * N + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] += __uint_as_float(w[i] << 16);
                acc[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[warp][lane * 8 + i] = acc[i];
    __syncthreads();
    const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (n < N) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kColWarps; ++w) s += sum[w][threadIdx.x];
        part[blockIdx.y * N + n] = s;
    }
}

__global__ void __launch_bounds__(256) colsum_join_kernel(const float* part, int64_t N, int splits,
                                                          __nv_bfloat16* out) {
    pdl_wait();
    pdl_trigger();
    const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int i = 0; i < splits; ++i) s += part[i * N + n];
    out[n] = __float2bfloat16_rn(s);
}

// Row ranges: about two CTAs per SM, at least 32 rows each.
int64_t col_splits(int64_t M, int64_t N) {
    const int64_t want = (2 * 148 * 256 + N - 1) / N, most = (M + 31) / 32;
    return want < 1 ? 1 : (want < most ? want : most);
}

}  // namespace

size_t colsum_bytes(int64_t M, int64_t N) { return size_t(col_splits(M, N)) * size_t(N) * 4; }

cudaError_t launch_colsum(const void* x, int64_t M, int64_t N, void* out, float* part, cudaStream_t st) {
    const int64_t s = col_splits(M, N), per = (M + s - 1) / s;
    const unsigned nb = unsigned((N + 255) / 256);
    cudaError_t e = launch_kernel(colsum_part_kernel, dim3(nb, unsigned(s)), dim3(kColWarps * 32), 0, st, true,
                                  (const __nv_bfloat16*)x, M, N, per, part);
    if (e != cudaSuccess) return e;
    return launch_kernel(colsum_join_kernel, dim3(nb), dim3(256), 0, st, true, (const float*)part, N, int(s),
                         (__nv_bfloat16*)out);
}

}  // namespace qmoe
