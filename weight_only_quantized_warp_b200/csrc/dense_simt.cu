// dense_simt.cu -- the products of the dense operators on fp32 FMAs: 64 x 64
// tiles, 16 k at a time through shared memory, 4 x 4 results a thread.
#include "dense.cuh"

namespace qmoe {
namespace {

constexpr int kT = 64, kKS = 16;

__device__ __forceinline__ float mx4_at(const DenseOperand& o, int64_t r, int64_t k, int64_t K) {
    const uint32_t b = reinterpret_cast<const uint8_t*>(o.p)[(r * K + k) >> 1];
    const uint32_t c = (k & 1) ? b >> 4 : b & 15u, e = (c >> 1) & 3u, m = c & 1u;
    const float mag = e == 0 ? 0.5f * float(m) : __uint_as_float(((e + 126u) << 23) | (m << 22));
    const uint32_t s = o.s[r * (K / 32) + k / 32];
    const float sc = __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
    return ((c & 8u) ? -mag : mag) * sc;
}

__global__ void __launch_bounds__(256) dense_simt_kernel(const DenseArgs a) {
    __shared__ float As[kKS][kT + 4], Bs[kKS][kT + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = int64_t(blockIdx.y) * kT, n0 = int64_t(blockIdx.x) * kT;
    float acc[4][4] = {};
    // pair order of the gated product: column 2i is gate i, 2i + 1 up i
    const bool split = a.epi == kEpiGate && !a.interleaved;
    for (int64_t k0 = 0; k0 < a.K; k0 += kKS) {
        for (int i = tid; i < kT * kKS; i += 256) {
            const int r = i / kKS, kk = i % kKS;
            const int64_t k = k0 + kk, m = m0 + r, n = n0 + r;
            float va = 0.0f, vb = 0.0f;
            if (k < a.K && m < a.M)
                va = a.mx4 ? mx4_at(a.a, m, k, a.K)
                           : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.a.p)[m * a.a.row + k * a.a.k_step]);
            if (k < a.K && n < a.N) {
                const int64_t nr = split ? (n >> 1) + (n & 1) * (a.N / 2) : n;
                vb = a.mx4 ? mx4_at(a.b, nr, k, a.K)
                           : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.b.p)[nr * a.b.row + k * a.b.k_step]);
            }
            As[kk][r] = va;
            Bs[kk][r] = vb;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kKS; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[kk][ty * 4 + i], Bs[kk][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= a.M) break;
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (n >= a.N) break;
            if (a.epi == kEpiStore) {
                if (a.out_f32)
                    ((float*)a.out)[m * a.N + n] = acc[i][j] + (a.bias ? ((const float*)a.bias)[n] : 0.0f);
                else
                    ((__nv_bfloat16*)a.out)[m * a.N + n] = __float2bfloat16_rn(
                        acc[i][j] + (a.bias ? __bfloat162float(((const __nv_bfloat16*)a.bias)[n]) : 0.0f));
            } else if (a.epi == kEpiGate) {
                if (j & 1) continue;
                const int64_t I = a.N / 2, c = n >> 1;
                const int64_t gi = a.interleaved ? n : c, ui = a.interleaved ? n + 1 : c + I;
                const __nv_bfloat16* b = (const __nv_bfloat16*)a.bias;
                const float g = acc[i][j] + (b ? __bfloat162float(b[gi]) : 0.0f);
                const float u = acc[i][j + 1] + (b ? __bfloat162float(b[ui]) : 0.0f);
                if (a.gu) {
                    a.gu[m * a.N + gi] = g;
                    a.gu[m * a.N + ui] = u;
                }
                ((__nv_bfloat16*)a.out)[m * I + c] = __float2bfloat16_rn(gate_value(a.gate, g, u));
            } else {
                const int64_t gi = m * 2 * a.N + (a.interleaved ? 2 * n : n);
                const int64_t ui = a.interleaved ? gi + 1 : gi + a.N;
                float hg, hu;
                const float h = gate_slopes(a.gate, a.gu[gi], a.gu[ui], hg, hu);
                ((__nv_bfloat16*)a.dgu)[gi] = __float2bfloat16_rn(acc[i][j] * hg);
                ((__nv_bfloat16*)a.dgu)[ui] = __float2bfloat16_rn(acc[i][j] * hu);
                ((__nv_bfloat16*)a.out)[m * a.N + n] = __float2bfloat16_rn(h);
            }
        }
    }
}

__global__ void __launch_bounds__(256) colsum_kernel(const __nv_bfloat16* x, int64_t M, int64_t N,
                                                     __nv_bfloat16* out) {
    const int64_t n = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int64_t m = 0; m < M; ++m) s += __bfloat162float(x[m * N + n]);
    out[n] = __float2bfloat16_rn(s);
}

}  // namespace

cudaError_t launch_dense(const DenseArgs& a, cudaStream_t st) {
    const dim3 grid(unsigned((a.N + kT - 1) / kT), unsigned((a.M + kT - 1) / kT));
    dense_simt_kernel<<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

size_t colsum_bytes(int64_t, int64_t) { return 0; }

cudaError_t launch_colsum(const void* x, int64_t M, int64_t N, void* out, float*, cudaStream_t st) {
    colsum_kernel<<<unsigned((N + 255) / 256), 256, 0, st>>>((const __nv_bfloat16*)x, M, N, (__nv_bfloat16*)out);
    return cudaGetLastError();
}

}  // namespace qmoe
