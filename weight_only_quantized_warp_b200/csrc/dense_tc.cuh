// dense_tc.cuh -- pieces of the dense operators' tcgen05 kernels beyond
// tc_common.cuh: CTA-pair and cluster PTX, operand descriptors for both
// majors and for 4-bit blocks, tensor maps and the epilogues' arithmetic.
#pragma once

#include <atomic>

#include "dense.cuh"
#include "tc_common.cuh"

namespace qmoe {
namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same shared-memory place in another CTA of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Bounded wait of one thread on a phase that the cluster's other CTAs complete
// (acquire at cluster scope). The clock is not read unless the first try fails.
__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.b32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                  int32_t* status, uint64_t limit_ns) {
    if (mbar_try_cluster(bar, parity)) return true;
    const uint64_t t0 = now_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (mbar_try_cluster(bar, parity)) return true;
        if ((spin & 15u) == 0u) {
            if (*abort_flag) return false;
            if (now_ns() - t0 > limit_ns) {
                *abort_flag = 1;
                atomicExch(status, int32_t(QMOE_TIMEOUT));
                return false;
            }
        }
    }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// TMA load by one CTA of a pair, completing on a barrier that may be the
// other CTA's (cluster address).
__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Arrive on the same barrier of both CTAs of the pair once the MMAs issued so
// far have completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "{\n.reg .b16 m;\nmov.b16 m, 3;\n"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ void mma_mx4_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sa,
                                             uint32_t sb, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(acc));
}

// 32 rows x 16 bytes of scales from shared memory to 4 tensor-memory columns
// of every lane quarter, in both CTAs of the pair.
__device__ __forceinline__ void cp_scales_pair(uint32_t t, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(t), "l"(sdesc) : "memory");
}

// The one-CTA forms.
__device__ __forceinline__ void mma_mx4_e(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sa,
                                          uint32_t sb, uint32_t acc, uint32_t e) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %6, 0;\nsetp.ne.b32 q, %7, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(e));
}
__device__ __forceinline__ void cp_scales_e(uint32_t t, uint64_t sdesc, uint32_t e) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}" ::"r"(t),
        "l"(sdesc), "r"(e)
        : "memory");
}
// Four floats to another CTA's shared memory (cluster address).
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}

// Shared-memory descriptor of an operand whose rows (M or N) lie along
// 128-byte swizzled lines of 64 bf16, one line per k: 64-row chunks 8192 bytes
// apart (64 k each), groups of 8 k 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn128(uint32_t saddr) {
    uint64_t d = uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t(8192 >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

// 512 bytes of scales: 32 rows of 16 bytes, unswizzled (8-row core matrices
// of 128 bytes, one after the other).
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
    uint64_t d = uint64_t((saddr >> 4) & 0x3FFFu);
    d |= uint64_t(1) << 16;
    d |= uint64_t(128 >> 4) << 32;
    d |= uint64_t(1) << 46;
    return d;
}

// Instruction descriptors. bf16: fp32 D, bf16 A and B, MN-major flags.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool amn, bool bmn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(amn) << 15) | (uint32_t(bmn) << 16) | (uint32_t(n >> 3) << 17) |
           (uint32_t(m >> 4) << 24);
}
// e2m1 A and B with E8M0 scales, taken from byte `id` (0 or 2) on of their words.
__host__ __device__ constexpr uint32_t idesc_mx4(int m, int n, int id) {
    return (uint32_t(id) << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (1u << 23) |
           (uint32_t(m >> 4) << 24) | (uint32_t(id) << 29);
}

// 32 accumulator columns of this warp's 32 lanes; tmem_wait_ld() before use.
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ---------------------------------------------------------------- host side

// Multiprocessors of the current device (looked up once per device).
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 2) return 148;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Raise a kernel's shared-memory limit, once per device.
template <auto Kern>
inline cudaError_t raise_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return e;
}

// Tensor map of up to three dimensions with 128-byte swizzled boxes (or
// plain ones): dims and boxes in elements, strides of the outer two in bytes.
struct MapSpec {
    const void* p;
    CUtensorMapDataType type;
    uint64_t dims[3], strides[2];
    uint32_t box[3];
    bool swizzle;
};

inline cudaError_t encode_map(CUtensorMap* map, const MapSpec& s) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {s.dims[0], s.dims[1], s.dims[2]}, strides[2] = {s.strides[0], s.strides[1]};
    const cuuint32_t box[3] = {s.box[0], s.box[1], s.box[2]}, es[3] = {1, 1, 1};
    return enc(map, s.type, 3, const_cast<void*>(s.p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               s.swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// Map of an operand (bf16): 128-byte boxes of `rows` rows along k, or 64 x 64
// boxes across. `pair` > 0: two row sets (gate, up) as the outer dimension,
// pair elements apart.
inline MapSpec bf16_spec(const DenseOperand& o, int64_t rows, int64_t K, uint32_t box_rows, int64_t pair) {
    MapSpec s{};
    s.p = o.p;
    s.type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    s.swizzle = true;
    const bool mn = o.k_step != 1;
    const int64_t line = mn ? o.k_step : o.row;
    s.dims[0] = uint64_t(mn ? rows : K);
    s.dims[1] = uint64_t(mn ? K : rows);
    s.dims[2] = pair ? 2 : 1;
    s.strides[0] = uint64_t(line) * 2;
    s.strides[1] = pair ? uint64_t(pair) * 2 : uint64_t(line) * 2;
    s.box[0] = 64;
    s.box[1] = mn ? 64 : box_rows;
    s.box[2] = 1;
    return s;
}

// Map of MX4 codes: 128-byte boxes (256 k) of `box_rows` rows.
inline MapSpec mx4_spec(const void* codes, int64_t rows, int64_t K, uint32_t box_rows) {
    MapSpec s{};
    s.p = codes;
    s.type = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    s.dims[0] = uint64_t(K / 2);
    s.dims[1] = uint64_t(rows);
    s.dims[2] = 1;
    s.strides[0] = s.strides[1] = uint64_t(K / 2);
    s.box[0] = 128;
    s.box[1] = box_rows;
    s.box[2] = 1;
    s.swizzle = true;
    return s;
}

}  // namespace
}  // namespace qmoe
