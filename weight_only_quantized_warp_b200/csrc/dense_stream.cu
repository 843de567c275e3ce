// dense_stream.cu -- the dense operators' products for few tokens (sm_100a).
//
// D[t, n] = sum_k X(t, k) W(n, k) for T <= 128 rows of X: bound by reading W
// once. W's rows are the MMA's M (128 of them, or 128 gate and 128 up rows as
// two accumulators) and the tokens its N, padded to NT = 16, 32, 64 or 128, so
// the tensor core takes both operands as they lie (MX4 codes undecoded) and
// the CTA does nothing per weight but move it: TMA fills a ring of 128-byte
// wide stages that an MMA warp empties. The backward pass's products (dh = dy w2,
// dx = dgu w1) run across the rows of W in memory: there a stage is 64 lines of
// 128 W columns and the descriptor says MN-major.
//
// K is split over the CTAs of a cluster so that about two CTAs per SM stream
// at once. Every rank finishes a range of tokens, in groups of four: the ranks
// store their fp32 partials of them into its shared memory (over the rings, once
// all have drained), 16 bytes a lane, and it adds them in rank order, so the
// result is the same on every call and there is no second launch. Loads of the
// other ranks' partials took a distributed-shared-memory latency per batch (3.5
// us of 8 at T = 64, N = K = 2048), 4-byte stores 2.5 us.
//
// MX4 scales are read where they lie: 128 threads (the later epilogue) take 32
// scales of a W row and of an X row at a time, four stages' worth, and place
// them for tcgen05.cp.
//
// Warps (192 threads): 0 TMA, 1 MMA and tensor memory, 2-5 scales and
// epilogue. Every wait is bounded (QMOE_TIMEOUT in the status word).
#include "dense_tc.cuh"

namespace qmoe {
namespace {

constexpr int kSThreads = 192;
constexpr int kSW = 128 * 128;  // W rows of a stage, one accumulator

struct StreamArgs {
    int64_t N, K;     // N: rows of W per accumulator (h columns for the gate)
    int T, nks, splits;
    int out_f32, interleaved, early_w;
    const uint8_t *ws, *xs;  // MX4 scales
    const void* bias;
    void* out;
    float* gu;             // kEpiGate: written when not null; kEpiGateBwd: read
    __nv_bfloat16* dgu;    // kEpiGateBwd
    float* sums;           // kEpiGateBwd: [splits, 2N] when not null
    GateParams gate;
    int32_t* status;
    int reset_status;
    DenseWaits waits;
};

__device__ uint32_t g_stream_gave_up;  // goes up, for every thread that leaves after an expired wait

template <bool MX4, bool GATE, int NT>
struct StreamCfg {
    static constexpr int kX = NT * 128;
    static constexpr int kS = MX4 ? 2048 : 0;  // W and X scales, 2 x 512 each
    static constexpr int kStage = kSW * (GATE ? 2 : 1) + kX + kS;
    // two CTAs per SM, but one where 128 tokens' gate and up partials need its memory
    static constexpr int kPerSm = GATE && NT == 128 ? 1 : 2;
    static constexpr int kStages = (kPerSm == 1 ? 200 : GATE ? 102 : 106) * 1024 / kStage;
    // partials, over the drained ring: up to 8 ranks' tokens padded to fours
    static constexpr int kPart = (NT + 32) * 512 * (GATE ? 2 : 1);
    static constexpr int kRing = kStages * kStage > kPart ? kStages * kStage : kPart;
    static constexpr int kSmem = kRing + 1024 + 1024;
    static constexpr int kAcc = NT * (GATE ? 2 : 1);
    static constexpr int kWant = kAcc + (MX4 ? 16 : 0);
    static constexpr int kCols = kWant <= 32 ? 32 : kWant <= 64 ? 64 : kWant <= 128 ? 128 : 256;
    static_assert(kStages >= 2 && kStage % 1024 == 0 && kSmem * kPerSm <= 226 * 1024, "shared memory");
    static_assert(kCols * kPerSm <= 512, "tensor memory");
};

// The results of W row n for up to NB tokens from t on, of which `left` exist:
// g (and u, for the gate) are their sums. kEpiGateBwd adds dgu to ag and au.
template <int EPI, int NB>
__device__ __forceinline__ void stream_emit(const StreamArgs& a, int t, int left, int64_t n,
                                            const float (&g)[NB], const float (&u)[NB], float bg, float bu, float& ag,
                                            float& au) {
    float sg[NB], su[NB];
    if (EPI == kEpiGateBwd) {  // all loads before any use
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const float* r = a.gu + int64_t(t + min(j, left - 1)) * 2 * a.N;
            asm volatile("ld.global.f32 %0, [%1];" : "=f"(sg[j]) : "l"(r + (a.interleaved ? 2 * n : n)));
            asm volatile("ld.global.f32 %0, [%1];" : "=f"(su[j]) : "l"(r + (a.interleaved ? 2 * n + 1 : a.N + n)));
        }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        if (j >= left) break;
        const int64_t tt = t + j;
        __nv_bfloat16* ob = reinterpret_cast<__nv_bfloat16*>(a.out) + tt * a.N + n;
        const int64_t gi = tt * 2 * a.N + (a.interleaved ? 2 * n : n), ui = a.interleaved ? gi + 1 : gi + a.N;
        if (EPI == kEpiGate) {
            const float vg = g[j] + bg, vu = u[j] + bu;
            if (a.gu) {
                a.gu[gi] = vg;
                a.gu[ui] = vu;
            }
            *ob = __float2bfloat16_rn(gate_value<-1, true>(a.gate, vg, vu));
        } else if (EPI == kEpiGateBwd) {
            float hg, hu;
            *ob = __float2bfloat16_rn(gate_slopes<-1, true>(a.gate, sg[j], su[j], hg, hu));
            const float dg = g[j] * hg, du = g[j] * hu;
            ag += dg;
            au += du;
            a.dgu[gi] = __float2bfloat16_rn(dg);
            a.dgu[ui] = __float2bfloat16_rn(du);
        } else if (a.out_f32) {
            reinterpret_cast<float*>(a.out)[tt * a.N + n] = g[j] + bg;
        } else {
            *ob = __float2bfloat16_rn(g[j] + bg);
        }
    }
}

template <bool MX4, int EPI, bool WMN, int NT>
__global__ void __launch_bounds__(kSThreads, StreamCfg<MX4, EPI == kEpiGate, NT>::kPerSm)
    dense_stream_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const StreamArgs a) {
    constexpr bool GATE = EPI == kEpiGate;
    using C = StreamCfg<MX4, GATE, NT>;
    constexpr int ST = C::kStages, KE = MX4 ? 128 : 64;  // map elements of a stage along k
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = a.splits > 1 ? int(cluster_rank()) : 0;
    const int n0 = int(blockIdx.x / a.splits) * 128;
    const int ks0 = int(int64_t(rank) * a.nks / a.splits), ks1 = int(int64_t(rank + 1) * a.nks / a.splits);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
    uint64_t* empty = full + ST;
    uint64_t* accf = empty + ST;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int first = min(ST, ks1 - ks0);  // stages in flight from the start
    auto load_w = [&](int ks, int s, uint32_t e) {
        const uint32_t sw = smem_u32(smem + s * C::kStage), fb = smem_u32(&full[s]);
        mbar_expect_tx_e(fb, C::kStage - C::kS, e);
        if (WMN) {
            tma_3d_e(sw, &wmap, n0, ks * 64, 0, fb, e);
            tma_3d_e(sw + 8192, &wmap, n0 + 64, ks * 64, 0, fb, e);
        } else {
            tma_3d_e(sw, &wmap, ks * KE, n0, 0, fb, e);
        }
        if (GATE) tma_3d_e(sw + kSW, &wmap, ks * KE, n0, 1, fb, e);
    };
    auto load_x = [&](int ks, int s, uint32_t e) {
        tma_3d_e(smem_u32(smem + s * C::kStage) + kSW * (GATE ? 2 : 1), &xmap, ks * KE, 0, 0, smem_u32(&full[s]), e);
    };
    if (warp == 0) {
        if (lane == 0) {
            for (int s = 0; s < ST; ++s) {
                mbar_init(smem_u32(&full[s]), MX4 ? 5 : 1);
                mbar_init(smem_u32(&empty[s]), 1);
            }
            mbar_init(smem_u32(accf), 1);
            *abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        // the first loads go out while the other warps set up; where W does not
        // depend on the kernel before this one, also while that one drains
        const uint32_t e = elect_one();
        if (!a.early_w) pdl_wait();
        for (int i = 0; i < first; ++i) load_w(ks0 + i, i, e);
        if (a.early_w) pdl_wait();
        for (int i = 0; i < first; ++i) load_x(ks0 + i, i, e);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    // not before the wait: the next kernel's early loads count on all that came
    // before this one being complete
    pdl_trigger();
    if (a.reset_status && blockIdx.x == 0 && tid == 32) *a.status = 0;

    if (warp == 0) {
        // ------------------------------------------------------- producer
        const uint32_t e = elect_one();
        int st = 0;
        uint32_t ph = 0;
        for (int ks = ks0 + first; ks < ks1; ++ks) {
            if (!warp_wait(smem_u32(&empty[st]), ph, abort_flag, a.status, a.waits.limit_ns)) break;
            load_w(ks, st, e);
            load_x(ks, st, e);
            if (++st == ST) { st = 0; ph ^= 1u; }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issue
        const uint32_t e = elect_one();
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        const uint32_t e_acc = a.waits.withhold ? 0u : e;
        const uint32_t ts = tmem + C::kAcc;  // scales: W chunk 0, 1, X chunk 0, 1 (4 columns each)
        for (int ks = ks0; ks < ks1; ++ks) {
            if (!warp_wait(smem_u32(&full[st]), ph, abort_flag, a.status, a.waits.limit_ns)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sw = smem_u32(smem + st * C::kStage), sx = sw + kSW * (GATE ? 2 : 1);
            const uint64_t wd = WMN ? desc_mn128(sw) : desc_sw128(sw), xd = desc_sw128(sx);
            const uint32_t acc0 = ks > ks0 ? 1u : 0u;
            if constexpr (MX4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) cp_scales_e(ts + 4 * j, desc_scales(sx + C::kX + 512 * j), e);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_mx4_e(tmem, wd + uint64_t(2 * kk), xd + uint64_t(2 * kk), idesc_mx4(128, NT, 2 * (kk & 1)),
                              ts + 4 * (kk >> 1), ts + 8 + 4 * (kk >> 1), kk > 0 ? 1u : acc0, e);
            } else {
                constexpr uint32_t id = idesc_f16(128, NT, WMN, false);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t acc = kk > 0 ? 1u : acc0;
                    mma_bf16_ss_e(tmem, wd + uint64_t((WMN ? 128 : 2) * kk), xd + uint64_t(2 * kk), id, acc, e);
                    if (GATE)
                        mma_bf16_ss_e(tmem + NT, desc_sw128(sw + kSW) + uint64_t(2 * kk), xd + uint64_t(2 * kk), id, acc, e);
                }
            }
            mma_commit_e(smem_u32(&empty[st]), e);
            if (++st == ST) { st = 0; ph ^= 1u; }
        }
        if (ok) mma_commit_e(smem_u32(accf), e_acc);
    } else {
        const int et = tid - 64;  // 0 .. 127
        bool ok = true;
        if constexpr (MX4) {
            // ------------------------------------------- scales: row et of W and X
            const int64_t pitch = a.K / 32, nw = n0 + et;
            int st = 0;
            uint32_t ph = 0;
            uint32_t w[8], x[8];
            auto fetch = [&](int ks) {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = x[j] = 0;
                if (ks >= ks1) return;
                if (nw < a.N) load_scales<8>(a.ws, a.N * pitch, nw, pitch, int64_t(ks) * 8, w);
                if (et < a.T) load_scales<8>(a.xs, int64_t(a.T) * pitch, et, pitch, int64_t(ks) * 8, x);
            };
            fetch(ks0);
            for (int ks = ks0; ok && ks < ks1; ks += 4) {
                uint32_t cw[8], cx[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) { cw[j] = w[j]; cx[j] = x[j]; }
                fetch(ks + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ks + i >= ks1) break;
                    ok = warp_wait(smem_u32(&empty[st]), ph ^ 1u, abort_flag, a.status, a.waits.limit_ns);
                    if (!ok) break;
                    uint32_t* sc = reinterpret_cast<uint32_t*>(smem + st * C::kStage + kSW + C::kX) +
                                   (et & 31) * 4 + (et >> 5);
                    sc[0] = cw[2 * i];
                    sc[128] = cw[2 * i + 1];
                    if (et < NT) {
                        sc[256] = cx[2 * i];
                        sc[384] = cx[2 * i + 1];
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&full[st]));
                    if (++st == ST) { st = 0; ph ^= 1u; }
                }
            }
        }
        // ------------------------------------------------------- epilogue
        ok = ok && warp_wait(smem_u32(accf), 0, abort_flag, a.status, a.waits.limit_ns);
        tc_fence_after();
        const int row = (warp & 3) * 32 + lane;
        const int64_t n = n0 + row;
        const bool valid = n < a.N;
        const uint32_t tb = tmem + (uint32_t((warp & 3) * 32) << 16);
        float bg = 0.0f, bu = 0.0f;
        if (a.bias && valid) {
            if (GATE) {
                const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(a.bias);
                bg = __bfloat162float(b[a.interleaved ? 2 * n : n]);
                bu = __bfloat162float(b[a.interleaved ? 2 * n + 1 : a.N + n]);
            } else {
                bg = a.out_f32 ? reinterpret_cast<const float*>(a.bias)[n]
                               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.bias)[n]);
            }
        }
        // partials at their owner: [rank][group of four tokens][accumulator][128 rows]
        constexpr int NACC = GATE ? 2 : 1;
        float4* part = reinterpret_cast<float4*>(smem);
        const int per = (a.T + 4 * a.splits - 1) / (4 * a.splits);  // groups of an owner
        if (a.splits > 1) {
            __syncwarp();
            cluster_sync_all();  // every ring has drained
        }
        float ag = 0.0f, au = 0.0f;  // kEpiGateBwd: over this rank's tokens
        if (ok) {
            const uint32_t mine = smem_u32(part + rank * per * NACC * 128 + row);
            int owner = 0, slot = 0;
            for (int t0 = 0; t0 < a.T; t0 += 16) {
                float v[16], u[16];
                tmem_ld16(tb + uint32_t(t0), v);
                if (GATE) tmem_ld16(tb + uint32_t(NT + t0), u);
                else for (int j = 0; j < 16; ++j) u[j] = 0.0f;
                if (a.splits > 1) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        if (t0 + j >= a.T) break;
                        const uint32_t to = map_rank(mine + uint32_t(slot * NACC * 2048), uint32_t(owner));
                        st_cluster_f32x4(to, v[j], v[j + 1], v[j + 2], v[j + 3]);
                        if (GATE) st_cluster_f32x4(to + 2048, u[j], u[j + 1], u[j + 2], u[j + 3]);
                        if (++slot == per) { slot = 0; ++owner; }
                    }
                } else if (valid) {
                    stream_emit<EPI, 16>(a, t0, a.T - t0, n, v, u, bg, bu, ag, au);
                }
                __syncwarp();
            }
        }
        if (a.splits > 1) {
            cluster_sync_all();  // every partial has arrived
            if (valid) {
                for (int q = 0; q < per && 4 * (rank * per + q) < a.T; ++q) {
                    const int t = 4 * (rank * per + q);
                    float g[4] = {}, u[4] = {};
                    for (int s = 0; s < a.splits; ++s) {
                        const float4* p = part + (s * per + q) * NACC * 128 + row;
                        const float4 x = p[0];
                        g[0] += x.x; g[1] += x.y; g[2] += x.z; g[3] += x.w;
                        if (GATE) {
                            const float4 y = p[128];
                            u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
                        }
                    }
                    stream_emit<EPI, 4>(a, t, a.T - t, n, g, u, bg, bu, ag, au);
                }
            }
        }
        if (EPI == kEpiGateBwd && a.sums && valid) {
            float* o = a.sums + int64_t(rank) * 2 * a.N;
            o[a.interleaved ? 2 * n : n] = ag;
            o[a.interleaved ? 2 * n + 1 : a.N + n] = au;
        }
    }
    if (a.splits > 1 && warp < 2) {
        __syncwarp();
        cluster_sync_all();
        cluster_sync_all();
    }
    __syncwarp();
    if (*abort_flag) {  // copies of the abandoned stages land before the memory goes away
        atomicAdd(&g_stream_gave_up, 1u);
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
    }
}

template <bool MX4, int EPI, bool WMN, int NT>
cudaError_t launch_nt(const CUtensorMap& wmap, const CUtensorMap& xmap, const StreamArgs& a, int tiles, cudaStream_t st) {
    constexpr auto kern = dense_stream_kernel<MX4, EPI, WMN, NT>;
    using C = StreamCfg<MX4, EPI == kEpiGate, NT>;
    cudaError_t e = raise_smem<kern>(C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(tiles * a.splits));
    cfg.blockDim = dim3(kSThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(a.splits);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, wmap, xmap, a);
}

template <bool MX4, int EPI, bool WMN>
cudaError_t launch_any(const CUtensorMap& wmap, const CUtensorMap& xmap, const StreamArgs& a, int tiles, cudaStream_t st) {
    if (a.T <= 16) return launch_nt<MX4, EPI, WMN, 16>(wmap, xmap, a, tiles, st);
    if (a.T <= 32) return launch_nt<MX4, EPI, WMN, 32>(wmap, xmap, a, tiles, st);
    if (a.T <= 64) return launch_nt<MX4, EPI, WMN, 64>(wmap, xmap, a, tiles, st);
    return launch_nt<MX4, EPI, WMN, 128>(wmap, xmap, a, tiles, st);
}

}  // namespace

cudaError_t dense_stream_gave_up(uint32_t* count, cudaStream_t st) {
    return cudaMemcpyFromSymbolAsync(count, g_stream_gave_up, sizeof *count, 0, cudaMemcpyDeviceToHost, st);
}

// Splits of K: as many (a cluster holds 8) as keep all CTAs resident and every
// split at least two stages long.
int64_t dense_stream_splits(const DenseArgs& d) {
    const bool gate = d.epi == kEpiGate;
    const int64_t tiles = ((gate ? d.N / 2 : d.N) + 127) / 128, nks = (d.K + (d.mx4 ? 255 : 63)) / (d.mx4 ? 256 : 64);
    const int64_t slots = (gate && d.M > 64 ? 1 : 2) * sm_count();
    int64_t splits = 1;
    while (splits < 8 && tiles * (splits + 1) <= slots && nks >= 2 * (splits + 1)) ++splits;
    return splits;
}

cudaError_t launch_dense_stream(const DenseArgs& d, bool early_w, cudaStream_t st) {
    const bool gate = d.epi == kEpiGate;
    StreamArgs a{};
    a.T = int(d.M);
    a.N = gate ? d.N / 2 : d.N;
    a.K = d.K;
    a.nks = int((d.K + (d.mx4 ? 255 : 63)) / (d.mx4 ? 256 : 64));
    a.out_f32 = d.out_f32;
    a.interleaved = d.interleaved;
    a.early_w = early_w;
    a.ws = d.b.s;
    a.xs = d.a.s;
    a.bias = d.bias;
    a.out = d.out;
    a.gu = d.gu;
    a.dgu = (__nv_bfloat16*)d.dgu;
    a.sums = d.sums;
    a.gate = d.gate;
    a.status = d.status;
    a.reset_status = d.reset_status;
    a.waits = dense_waits();
    const int64_t tiles = (a.N + 127) / 128;
    a.splits = int(dense_stream_splits(d));
    if (tiles * a.splits > (int64_t(1) << 30)) return cudaErrorInvalidValue;
    const uint32_t nt = d.M <= 16 ? 16 : d.M <= 32 ? 32 : d.M <= 64 ? 64 : 128;
    CUtensorMap wmap, xmap;
    cudaError_t e;
    if (d.mx4) {
        if ((e = encode_map(&wmap, mx4_spec(d.b.p, d.N, d.K, 128))) != cudaSuccess) return e;
        if ((e = encode_map(&xmap, mx4_spec(d.a.p, d.M, d.K, nt))) != cudaSuccess) return e;
        return launch_any<true, kEpiStore, false>(wmap, xmap, a, int(tiles), st);
    }
    if ((e = encode_map(&xmap, bf16_spec(d.a, d.M, d.K, nt, 0))) != cudaSuccess) return e;
    DenseOperand w = d.b;
    if (gate && d.interleaved) w.row *= 2;
    e = encode_map(&wmap, bf16_spec(w, a.N, d.K, 128, !gate ? 0 : d.interleaved ? d.b.row : a.N * d.b.row));
    if (e != cudaSuccess) return e;
    if (gate) return launch_any<false, kEpiGate, false>(wmap, xmap, a, int(tiles), st);
    if (d.epi == kEpiGateBwd) return launch_any<false, kEpiGateBwd, true>(wmap, xmap, a, int(tiles), st);
    return d.b.k_step != 1 ? launch_any<false, kEpiStore, true>(wmap, xmap, a, int(tiles), st)
                           : launch_any<false, kEpiStore, false>(wmap, xmap, a, int(tiles), st);
}

}  // namespace qmoe
