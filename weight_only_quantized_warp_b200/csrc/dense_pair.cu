// dense_pair.cu -- the dense operators' products on tcgen05 CTA pairs (sm_100a).
//
// D[m, n] = sum_k A(m, k) B(n, k). Two CTAs of a cluster work on one 256 x BN
// tile (cta_group::2): each loads its 128 rows of A and its half of B's rows,
// so a tile's operand bytes per MAC are half of what a single CTA with the
// same accumulators would load, and accumulates its 128 rows x BN columns in
// tensor memory. Two accumulators alternate, so the epilogue of one tile runs
// under the MMAs of the next. Tiles are walked in groups of kGroupM tile rows
// by all columns, so that the operands of the tiles in flight stay in L2.
//
// Operands come by TMA in stages of 128 bytes of k per row (64 bf16 or 256
// e2m1) into 128-byte swizzled lines; ends of M, N and K are zero-filled by
// the copies. Where the reduction runs across the rows of a matrix in memory
// (the backward pass: w2 and w1 as B of dh and dx, all operands of the weight
// gradients) the stage is 64 k lines of 64 rows and the descriptor says
// MN-major; nothing is transposed in memory.
//
// kind::mxf4 (MX4): products of e2m1 values with both E8M0 scales applied by
// the tensor core, two scales per row and MMA (64 k). Scales are copied with
// each stage from an array tiled beforehand (ScaleTiles) and from shared
// to tensor memory by tcgen05.cp ahead of the stage's MMAs. BN is 240, not
// 256: two 240-column accumulators leave 32 columns for a stage's scales.
//
// Gate epilogue: B's first half of a tile is 128 gate rows and the second 128
// up rows (one per CTA), so a thread holds gate and up of the same column.
//
// Warps (384 threads): 0 TMA, 1 MMA issue (leader CTA) and tensor memory, one
// thread of each issuing; 4-11 epilogue. Every wait is bounded (then
// QMOE_TIMEOUT in the status word, every role leaves its loop).
#include "dense_tc.cuh"

namespace qmoe {
namespace {

constexpr int kPThreads = 384;
constexpr int kPEpi0 = 4, kPEpiWarps = 8;
constexpr int kGroupM = 8;  // 2, 4 and 16 measured the same
constexpr int kABytes = 128 * 128;  // one CTA's A rows of a stage

// One product of a launch.
struct PairProblem {
    int64_t M, N;          // N: result columns (h columns for the gate)
    int tiles_m, tiles_n, nks;
    int bn;                // columns of a tile (accumulators, both halves)
    int amn;               // A lies MN-major (launches of several products)
    int early_b;           // B was not written by the kernel before this one
    int vec_out;
    void* out;
};

// A launch walks up to three products: the tiles of p[0], then those of p[1] and
// p[2] as one list (the backward pass's dx, and dw1 and dw2, which are shorter).
struct PairArgs {
    PairProblem p[3];
    int tiles[3];
    int head;              // see tile_at
    int chunks;
    int out_f32, interleaved;
    const void* bias;
    float* gu;
    void* dgu;
    float* sums;           // see DenseArgs
    GateParams gate;
    int32_t* status;
    int reset_status;
    DenseWaits waits;
};

__device__ uint32_t g_pair_gave_up;  // goes up, for every thread that leaves after an expired wait

struct PairMaps {
    CUtensorMap a[3], b[3];  // MX4: a[1], b[1] are the tiled scales
};

template <bool MX4>
struct PairCfg {
    static constexpr int BN = MX4 ? 240 : 256;
    static constexpr int kB = BN / 2 * 128;
    static constexpr int kSA = MX4 ? 1024 : 0, kSB = MX4 ? 2048 : 0;
    static constexpr int kStage = kABytes + kB + kSA + kSB;
    static constexpr int kStages = MX4 ? 5 : 6;
    static constexpr int kTurnOff = kStages * kStage;         // 4 KB per epilogue warp
    static constexpr int kBarOff = kTurnOff + kPEpiWarps * 4096;
    static constexpr int kSmem = kBarOff + 1024 + 1024;
    static_assert(kStage % 1024 == 0 && kSmem <= 227 * 1024, "stages");
};

// The i-th tile of a pair. p[0]'s tiles go round the pairs. Where they do not
// come out even, the pairs left with one fewer start on the second list `head`
// of its tiles early (as many as take the time of one of p[0]'s), and the rest
// of that list goes round all pairs.
template <bool MULTI>
__device__ __forceinline__ bool tile_at(const PairArgs& a, int i, int& q, int& tm, int& tn) {
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, D = a.tiles[0], W = a.tiles[1] + a.tiles[2];
    int t = pair + i * pairs;
    q = 0;
    if (t >= D) {
        if (!MULTI || W == 0) return false;
        const int r = D % pairs, E = r ? pairs - r : 0, base = min(W, E * a.head);
        i -= pair < D ? (D - 1 - pair) / pairs + 1 : 0;
        t = base + pair + i * pairs;
        if (E && pair >= r) t = i < a.head ? pair - r + i * E : t - a.head * pairs;
        if (t >= (E && pair >= r && i < a.head ? base : W)) return false;
        q = t < a.tiles[1] ? 1 : 2;
        if (q == 2) t -= a.tiles[1];
    }
    const PairProblem& p = a.p[MULTI ? q : 0];
    const int per = kGroupM * p.tiles_n;
    const int g = t / per, m0 = g * kGroupM, gm = min(p.tiles_m - m0, kGroupM), rr = t - g * per;
    tm = m0 + rr % gm;
    tn = rr / gm;
    return true;
}

// 32 accumulator columns of the warp's lanes (columns past the tile's are read
// too, inside the allocation, and not used).
__device__ __forceinline__ void tmem_f32(uint32_t t, float (&v)[32]) {
    uint32_t r[32];
    tmem_ld32(t, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Turn of a block of 32 rows through a warp's 4 KB: in tensor memory a lane
// holds a row, in global memory a row wants neighbouring lanes. A row is NU
// units of 16 bytes (8: 32 fp32 or 64 bf16 columns; 4: 32 bf16). Lane r writes
// row r; then NU lanes read a row's units and 32 / NU rows go out in one
// instruction. Unit j of row r lies at place j ^ (r NU / 8 mod NU) of its line:
// eight neighbouring lanes hit eight different 16-byte banks both ways.
template <int NU>
__device__ __forceinline__ int turn_at(int row, int j) {
    return row * NU + (j ^ ((row * NU / 8) & (NU - 1)));
}
template <int NU>
__device__ __forceinline__ void turn_put(uint4* buf, int lane, const uint4 (&v)[NU]) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NU; ++j) buf[turn_at<NU>(lane, j)] = v[j];
    __syncwarp();
}
__device__ __forceinline__ void put_f32(uint4* buf, int lane, const float (&v)[32]) {
    uint4 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w[j] = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                          __float_as_uint(v[4 * j + 3]));
    turn_put<8>(buf, lane, w);
}
__device__ __forceinline__ void pack32(const float (&v)[32], uint4* w) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                          pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
}

// A turned block to rows of `ld` elements: `rows` of its rows, `cols` of its
// columns; out is at its first element. vec: rows start on 16 bytes.
// Otherwise (eight units) lanes take words of a row, whole where those are
// aligned.
template <int NU, typename T>
__device__ __forceinline__ void turn_out(const uint4* buf, T* out, int64_t ld, int rows, int cols, bool vec, int lane) {
    constexpr int E = 16 / int(sizeof(T)), RI = 32 / NU;
    if (NU != 8 || vec) {
        const int j = lane % NU, r0 = lane / NU;
        T* o = out + r0 * ld + j * E;
        const bool mine = j * E < cols;  // cols is a multiple of E where rows are aligned
        uint4 v[NU];
#pragma unroll
        for (int i = 0; i < NU; ++i) v[i] = buf[turn_at<NU>(i * RI + r0, j)];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            if (mine && i * RI + r0 < rows) *reinterpret_cast<uint4*>(o) = v[i];
            o += RI * ld;
        }
        return;
    }
    if constexpr (NU == 8) {  // a line is 32 words, one a lane
        const uint32_t* words = reinterpret_cast<const uint32_t*>(buf);
        constexpr int EW = 4 / int(sizeof(T));  // elements of a word
        const bool whole = EW == 1 || (((reinterpret_cast<uintptr_t>(out) & 3) == 0) && ld % 2 == 0);
        T* o = out + lane * EW;
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 8) {
            uint32_t v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = words[turn_at<NU>(r0 + r, lane >> 2) * 4 + (lane & 3)];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r0 + r < rows) {
                    if (lane * EW + EW <= cols && whole) {
                        *reinterpret_cast<uint32_t*>(o) = v[r];
                    } else if (EW == 2) {
                        if (2 * lane < cols) reinterpret_cast<uint16_t*>(o)[0] = uint16_t(v[r]);
                        if (2 * lane + 1 < cols) reinterpret_cast<uint16_t*>(o)[1] = uint16_t(v[r] >> 16);
                    }
                }
                o += ld;
            }
        }
    }
}

// Loads that stay where they are written, ahead of the arithmetic: a batch of
// them covers one latency.
__device__ __forceinline__ float4 ld_early(const float* p) {
    float4 v;
    asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// MULTI: several products, whose A lies as each says; else A lies along k. BMN: B
// lies across its rows.
template <bool MX4, bool MULTI, bool BMN, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPThreads, 1)
    dense_pair_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairArgs a) {
    using C = PairCfg<MX4>;
    constexpr int ST = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    // the dynamic segment starts at the same address in both CTAs, so the
    // aligned offsets agree
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + ST;
    uint64_t* accf = empty + ST;
    uint64_t* acce = accf + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&accf[b]), 1);
            mbar_init(smem_u32(&acce[b]), 2 * kPEpiWarps);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 64) {
        for (int i = 0; i < (MULTI ? 3 : MX4 ? 2 : 1); ++i) {
            if (MULTI && a.tiles[i] == 0) continue;
            prefetch_map(&maps.a[i]);
            prefetch_map(&maps.b[i]);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp != 0) {  // everything up to here touched no global memory
        pdl_wait();
        pdl_trigger();
    }
    if (a.reset_status && blockIdx.x == 0 && tid == 32) *a.status = 0;

    if (warp == 0) {
        // ------------------------------------------------------- producer
        // one thread: a stage's turn (wait, expect, two to four copies) has to
        // take less than its MMAs, 320 clocks at 160 columns
        if (elect_one()) {
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            const uint32_t stage0 = smem_u32(smem), full0 = map_rank(smem_u32(full), 0);  // the leader's barriers
            auto load_b = [&](int q, int tn, int ks, int s) {
                const int BN = a.p[MULTI ? q : 0].bn;
                const uint32_t sb = stage0 + s * C::kStage + kABytes, fb = full0 + 8 * s;
                const int n0 = EPI == kEpiGate ? tn * (BN / 2) : tn * BN + int(rank) * (BN / 2);
                // bytes of both CTAs' copies of a stage
                if (rank == 0)
                    mbar_expect_tx(smem_u32(full) + 8 * s,
                                   2u * uint32_t(kABytes + (BMN ? (BN > 128 ? 16384 : 8192) : BN * 64) +
                                                 (MX4 ? C::kSA + (BN > 128 ? C::kSB : C::kSB / 2) : 0)));
                const CUtensorMap* m = &maps.b[MULTI ? q : 0];
                if (BMN) {
                    tma_3d_pair(sb, m, n0, ks * 64, 0, fb);
                    if (BN > 128) tma_3d_pair(sb + 8192, m, n0 + 64, ks * 64, 0, fb);
                } else {
                    tma_3d_pair(sb, m, ks * (MX4 ? 128 : 64), n0, EPI == kEpiGate ? int(rank) : 0, fb);
                }
            };
            auto load_a = [&](int q, int tm, int tn, int ks, int s) {
                const uint32_t sa = stage0 + s * C::kStage, fb = full0 + 8 * s;
                const int m0 = tm * 256 + int(rank) * 128;
                const CUtensorMap* m = &maps.a[MULTI ? q : 0];
                if (MULTI && a.p[MULTI ? q : 0].amn) {
                    tma_3d_pair(sa, m, m0, ks * 64, 0, fb);
                    tma_3d_pair(sa + 8192, m, m0 + 64, ks * 64, 0, fb);
                } else {
                    tma_3d_pair(sa, m, ks * (MX4 ? 128 : 64), m0, 0, fb);
                }
                if (MX4) {
                    const uint32_t ss = sa + kABytes + C::kB;
                    tma_3d_pair(ss, &maps.a[1], 0, (m0 >> 7) * a.chunks + 2 * ks, 0, fb);
                    // rows of 512 bytes: a chunk of up to 128 tile rows
                    tma_3d_pair(ss + C::kSA, &maps.b[1], 0, (tn * a.chunks + 2 * ks) * (a.p[0].bn > 128 ? 2 : 1), 0, fb);
                }
            };
            int ks = 0, q, tm, tn;
            const bool any = tile_at<MULTI>(a, 0, q, tm, tn);
            if (any && a.p[MULTI ? q : 0].early_b) {
                // the first stages of B while the kernel before this one drains
                const int first = min(ST, a.p[MULTI ? q : 0].nks);
                for (int i = 0; i < first; ++i) load_b(q, tn, i, i);
                pdl_wait();
                for (; ks < first; ++ks) load_a(q, tm, tn, ks, ks);
                if (first == ST) ph = 1;
                else st = first;
            } else {
                pdl_wait();
            }
            for (int i = 0; ok && tile_at<MULTI>(a, i, q, tm, tn); ++i) {
                for (; ks < a.p[MULTI ? q : 0].nks; ++ks) {
                    ok = mbar_wait(smem_u32(&empty[st]), ph ^ 1u, abort_flag, a.status, a.waits.limit_ns);
                    if (!ok) break;
                    load_b(q, tn, ks, st);
                    load_a(q, tm, tn, ks, st);
                    if (++st == ST) { st = 0; ph ^= 1u; }
                }
                ks = 0;
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------- MMA issue
        if (elect_one()) {
            int st = 0, acc = 0;
            uint32_t ph = 0, cph = 0;
            bool ok = true;
            const uint32_t tscale = tmem + 2 * C::BN;  // MX4: A chunk 0, 1 (4 columns each), B chunk 0, 1 (8 each)
            int q, tm, tn;
            for (int i = 0; ok && tile_at<MULTI>(a, i, q, tm, tn); ++i) {
                if (!mbar_wait_cluster(smem_u32(&acce[acc]), cph ^ 1u, abort_flag, a.status, a.waits.limit_ns)) break;
                tc_fence_after();
                const int BN = a.p[MULTI ? q : 0].bn, nks = a.p[MULTI ? q : 0].nks;
                const bool amn = MULTI && a.p[MULTI ? q : 0].amn;
                const uint32_t idesc = idesc_f16(256, BN, amn, BMN);
                const uint32_t d = tmem + uint32_t(acc * C::BN);
                for (int ks = 0; ks < nks; ++ks) {
                    ok = mbar_wait_cluster(smem_u32(&full[st]), ph, abort_flag, a.status, a.waits.limit_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + st * C::kStage), sb = sa + kABytes;
                    const uint32_t acc0 = ks > 0 ? 1u : 0u;
                    if constexpr (MX4) {
                        const uint32_t ssa = sb + C::kB, ssb = ssa + C::kSA;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            cp_scales_pair(tscale + 4 * j, desc_scales(ssa + 512 * j));
                            cp_scales_pair(tscale + 8 + 8 * j, desc_scales(ssb + (BN > 128 ? 1024 : 512) * j));
                            if (BN > 128) cp_scales_pair(tscale + 12 + 8 * j, desc_scales(ssb + 1024 * j + 512));
                        }
                        const uint64_t ad = desc_sw128(sa), bd = desc_sw128(sb);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_mx4_pair(d, ad + uint64_t(2 * kk), bd + uint64_t(2 * kk), idesc_mx4(256, BN, 2 * (kk & 1)),
                                           tscale + 4 * (kk >> 1), tscale + 8 + 8 * (kk >> 1), kk > 0 ? 1u : acc0);
                    } else {
                        const uint64_t ad = amn ? desc_mn128(sa) : desc_sw128(sa);
                        const uint64_t bd = BMN ? desc_mn128(sb) : desc_sw128(sb);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)  // 16 k: 32 bytes into each line, or 16 lines on
                            mma_bf16_pair(d, ad + uint64_t((amn ? 128 : 2) * kk), bd + uint64_t((BMN ? 128 : 2) * kk),
                                            idesc, kk > 0 ? 1u : acc0);
                    }
                    mma_commit_pair(smem_u32(&empty[st]));
                    if (++st == ST) { st = 0; ph ^= 1u; }
                }
                if (!ok) break;
                if (i > 0 || !a.waits.withhold) mma_commit_pair(smem_u32(&accf[acc]));
                if (++acc == 2) { acc = 0; cph ^= 1u; }
            }
        }
    } else if (warp >= kPEpi0) {
        // ------------------------------------------------------- epilogue
        const int qd = warp & 3, half = (warp - kPEpi0) >> 2;
        uint4* turn = reinterpret_cast<uint4*>(smem + C::kTurnOff + (warp - kPEpi0) * 4096);
        int acc = 0;
        uint32_t cph = 0;
        int q, tm, tn;
        for (int i = 0; tile_at<MULTI>(a, i, q, tm, tn); ++i) {
            const PairProblem& p = a.p[MULTI ? q : 0];
            const int64_t M = p.M, N = p.N;
            const int BN = p.bn;
            const int64_t m0 = int64_t(tm) * 256 + rank * 128 + qd * 32;
            const int rows = int(max(int64_t(0), min(int64_t(32), M - m0)));
            const int64_t end = min(N, int64_t(tn + 1) * (EPI == kEpiGate ? BN / 2 : BN));
            if (!warp_wait(smem_u32(&accf[acc]), cph, abort_flag, a.status, a.waits.limit_ns)) break;
            tc_fence_after();
            const uint32_t tb = tmem + (uint32_t(qd * 32) << 16) + uint32_t(acc * C::BN);
            if (EPI == kEpiStore) {
                // 32 columns with the bias of theirs
                auto fetch = [&](int c, int64_t n, float (&v)[32]) {
                    tmem_f32(tb + uint32_t(c), v);
                    if (a.bias) {
                        const float b = n + lane >= end ? 0.0f
                                        : a.out_f32     ? ((const float*)a.bias)[n + lane]
                                                        : __bfloat162float(((const __nv_bfloat16*)a.bias)[n + lane]);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, b, i);
                    }
                };
                float v[32];
                if (a.out_f32) {
                    for (int c = half * 32; c < BN; c += 64) {
                        const int64_t n = int64_t(tn) * BN + c;
                        if (n >= end) break;  // uniform over the warp
                        fetch(c, n, v);
                        put_f32(turn, lane, v);
                        turn_out<8>(turn, (float*)p.out + m0 * N + n, N, rows, int(min(int64_t(32), end - n)), p.vec_out,
                                    lane);
                    }
                } else {
                    for (int c = half * 64; c < BN; c += 128) {
                        const int64_t n = int64_t(tn) * BN + c;
                        if (n >= end) break;
                        uint4 w[8];
                        fetch(c, n, v);
                        pack32(v, w);
                        if (n + 32 < end) {
                            fetch(c + 32, n + 32, v);
                            pack32(v, w + 4);
                        }
                        turn_put<8>(turn, lane, w);
                        turn_out<8>(turn, (__nv_bfloat16*)p.out + m0 * N + n, N, rows, int(min(int64_t(64), end - n)),
                                    p.vec_out, lane);
                    }
                }
            } else if (EPI == kEpiGate) {
                const int bh = BN / 2;
                for (int c = half * 32; c < bh; c += 64) {
                    const int64_t n = int64_t(tn) * bh + c;
                    if (n >= end) break;
                    const int cols = int(min(int64_t(32), end - n));  // a multiple of 8, as N and bh are
                    float g[32], u[32];
                    tmem_f32(tb + uint32_t(c), g);
                    tmem_f32(tb + uint32_t(bh + c), u);
                    if (a.bias) {
                        const __nv_bfloat16* b = (const __nv_bfloat16*)a.bias;
                        float bg = 0.0f, bu = 0.0f;
                        if (lane < cols) {
                            bg = __bfloat162float(b[a.interleaved ? 2 * (n + lane) : n + lane]);
                            bu = __bfloat162float(b[a.interleaved ? 2 * (n + lane) + 1 : N + n + lane]);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            g[i] += __shfl_sync(0xffffffffu, bg, i);
                            u[i] += __shfl_sync(0xffffffffu, bu, i);
                        }
                    }
                    if (a.gu) {
                        float* gr = a.gu + m0 * 2 * N;
                        if (a.interleaved) {
#pragma unroll
                            for (int k = 0; k < 32; k += 16) {
                                float w[32];
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    w[2 * i] = g[k + i];
                                    w[2 * i + 1] = u[k + i];
                                }
                                put_f32(turn, lane, w);
                                turn_out<8>(turn, gr + 2 * (n + k), 2 * N, rows, 2 * (cols - k), true, lane);
                            }
                        } else {
                            put_f32(turn, lane, g);
                            turn_out<8>(turn, gr + n, 2 * N, rows, cols, true, lane);
                            put_f32(turn, lane, u);
                            turn_out<8>(turn, gr + N + n, 2 * N, rows, cols, true, lane);
                        }
                    }
                    with_gate_mode(a.gate, [&](auto mode) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            g[i] = gate_value<decltype(mode)::value, decltype(mode)::clamp>(a.gate, g[i], u[i]);
                    });
                    uint4 w[4];
                    pack32(g, w);
                    turn_put<4>(turn, lane, w);
                    turn_out<4>(turn, (__nv_bfloat16*)p.out + m0 * N + n, N, rows, cols, true, lane);
                }
            } else {
                // dh turned to eight lanes a row, four columns each, beside g and
                // u, which are loaded four steps (of four rows) ahead of their use:
                // slot k of the unrolled loop always holds the same registers, so
                // that no move waits for a load.
                const int j = lane & 7, r0 = lane >> 3;
                const int64_t c0 = int64_t(tn) * BN + half * 32 + 4 * j;
                const int steps = 8 * int((max(int64_t(0), end - (c0 - 4 * j)) + 63) / 64);
                const int64_t apart = a.interleaved ? 4 : N;  // of g, u, g, u, ... or of fours of g and of u
                // step s: rows 4 (s % 8) + r0 of the block at column c0 + 64 (s / 8);
                // past the matrix the last row or column that there is
                auto load_gu = [&](int s, float4& x, float4& y) {
                    const int64_t col = min(c0 + 64 * (s >> 3), N - 4), row = min(m0 + r0 + 4 * (s & 7), M - 1);
                    const float* r = a.gu + row * 2 * N + (a.interleaved ? 2 * col : col);
                    x = ld_early(r);
                    y = ld_early(r + apart);
                };
                with_gate_mode(a.gate, [&](auto mode) {
                    float4 xs[4], ys[4];
                    float ag[4], au[4];  // the lane's columns over the block's rows
#pragma unroll
                    for (int k = 0; k < 4; ++k) load_gu(k, xs[k], ys[k]);
#pragma unroll 1
                    for (int s0 = 0; s0 < steps; s0 += 4) {
                        if ((s0 & 7) == 0) {
                            float v[32];
                            tmem_f32(tb + uint32_t(half * 32 + 8 * s0), v);
                            put_f32(turn, lane, v);
#pragma unroll
                            for (int k = 0; k < 4; ++k) ag[k] = au[k] = 0.0f;
                        }
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const int s = s0 + k4;
                            const uint4 w = turn[turn_at<8>(4 * (s & 7) + r0, j)];
                            const float4 x = xs[k4], y = ys[k4];
                            const float dh[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                                                 __uint_as_float(w.w)};
                            const float g[4] = {x.x, a.interleaved ? x.z : x.y, a.interleaved ? y.x : x.z,
                                                a.interleaved ? y.z : x.w};
                            const float u[4] = {a.interleaved ? x.y : y.x, a.interleaved ? x.w : y.y,
                                                a.interleaved ? y.y : y.z, y.w};
                            float h[4], dg[4], du[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float hg, hu;
                                h[k] = gate_slopes<decltype(mode)::value, decltype(mode)::clamp>(a.gate, g[k], u[k],
                                                                                                 hg, hu);
                                dg[k] = dh[k] * hg;
                                du[k] = dh[k] * hu;
                            }
                            const int64_t col = c0 + 64 * (s >> 3);
                            if (4 * (s & 7) + r0 < rows && col < end) {  // N is a multiple of 8: whole fours
                                const int64_t row = m0 + r0 + 4 * (s & 7);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    ag[k] += dg[k];
                                    au[k] += du[k];
                                }
                                *reinterpret_cast<uint2*>((__nv_bfloat16*)p.out + row * N + col) =
                                    make_uint2(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]));
                                const int64_t at = row * 2 * N + (a.interleaved ? 2 * col : col);
                                __nv_bfloat16* d = (__nv_bfloat16*)a.dgu + at;
                                if (a.interleaved) {
                                    *reinterpret_cast<uint4*>(d) =
                                        make_uint4(pack_bf16(dg[0], du[0]), pack_bf16(dg[1], du[1]),
                                                   pack_bf16(dg[2], du[2]), pack_bf16(dg[3], du[3]));
                                } else {
                                    *reinterpret_cast<uint2*>(d) =
                                        make_uint2(pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3]));
                                    *reinterpret_cast<uint2*>(d + N) =
                                        make_uint2(pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3]));
                                }
                            }
                            load_gu(min(s + 4, steps - 1), xs[k4], ys[k4]);
                        }
                        if ((s0 & 4) && a.sums) {
                            // Each of the four lanes of the same columns ends with one column's g
                            // and u (all four sums in each lane, and whole vectors to store, took
                            // registers that spilled: a training step 149.8 against 149.1 us).
                            const bool hi = lane & 16, odd = lane & 8;
                            auto join = [&](const float (&v)[4]) {
                                const float x = (hi ? v[2] : v[0]) + __shfl_xor_sync(~0u, hi ? v[0] : v[2], 16);
                                const float y = (hi ? v[3] : v[1]) + __shfl_xor_sync(~0u, hi ? v[1] : v[3], 16);
                                return (odd ? y : x) + __shfl_xor_sync(~0u, odd ? x : y, 8);
                            };
                            const float sg = join(ag), su = join(au);
                            const int64_t col = c0 + 64 * (s0 >> 3) + (hi ? 2 : 0) + (odd ? 1 : 0);
                            if (rows > 0 && col < end) {
                                float* o = a.sums + (m0 >> 5) * 2 * N;
                                o[a.interleaved ? 2 * col : col] = sg;
                                o[a.interleaved ? 2 * col + 1 : N + col] = su;
                            }
                        }
                        __syncwarp();
                    }
                });
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&acce[acc]), 0));
            if (++acc == 2) { acc = 0; cph ^= 1u; }
        }
    }

    __syncwarp();
    if (*abort_flag) {  // copies of the abandoned stages land before the memory goes away
        atomicAdd(&g_pair_gave_up, 1u);
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

template <bool MX4, bool MULTI, bool BMN, int EPI>
cudaError_t launch_one(const PairMaps& maps, PairArgs& a, cudaStream_t st) {
    a.waits = dense_waits();
    constexpr auto kern = dense_pair_kernel<MX4, MULTI, BMN, EPI>;
    cudaError_t e = raise_smem<kern>(PairCfg<MX4>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = int64_t(a.tiles[0]) + a.tiles[1] + a.tiles[2], pairs = sm_count() / 2;
    const int grid = 2 * int(tiles < pairs ? tiles : pairs);
    return launch_kernel(kern, dim3(unsigned(grid)), dim3(kPThreads), PairCfg<MX4>::kSmem, st, true, maps, a);
}

// Tile columns: the widest (256; 240 for MX4) where the tiles fill many rounds
// of the 74 pairs. With few rounds a narrower tile can save a large part of the
// last, half-empty one: the width (a multiple of 32, at least 128) with the
// smallest rounds x (BN + 256), a stage's operand bytes per CTA, which is what a
// stage takes below 256 columns. Measured at T = 1024, H = I = 2880 (160
// columns) against 256 throughout: forward 46 against 56 us, training step 148
// against 158; 160 columns at T = 4096, H = 4096, I = 14336 (where the rule
// keeps 256) take 4080 us against 3390. MX4 at T = 1001, N = 2817 (160 columns)
// against 240: 13.3 against 15.0 us.
// A second product of the same launch counts its tiles too. The 74 pairs of a
// B200 are planned for whatever the device has, because the size of a workspace
// follows from the width and is asked for without a device.
int pair_width(int64_t tiles_m, int64_t n, bool mx4, int64_t tiles_m2 = 0, int64_t n2 = 0) {
    constexpr int64_t kPairs = 74;
    int best = 0;
    int64_t cost = INT64_MAX;
    for (int bn = mx4 ? PairCfg<true>::BN : 256; bn >= 128; bn = (bn - 1) / 32 * 32) {
        const int64_t tiles = tiles_m * ((n + bn - 1) / bn) + tiles_m2 * ((n2 + bn - 1) / bn);
        const int64_t c = (tiles + kPairs - 1) / kPairs * (bn + 256);
        if (c < cost) {
            cost = c;
            best = bn;
        }
    }
    return best;
}

int64_t pair_chunks(int64_t K) { return 2 * ((K + 255) / 256); }
int64_t up256(int64_t v) { return (v + 255) & ~int64_t(255); }

}  // namespace

cudaError_t dense_pair_gave_up(uint32_t* count, cudaStream_t st) {
    return cudaMemcpyFromSymbolAsync(count, g_pair_gave_up, sizeof *count, 0, cudaMemcpyDeviceToHost, st);
}

void dense_pair_tiles(int64_t M, int64_t N, int64_t K, void* scratch, ScaleTiles* a, ScaleTiles* b) {
    const int BN = pair_width((M + 255) / 256, N, true);
    *a = {nullptr, (uint8_t*)scratch, M, 128, int((M + 255) / 256) * 2, int(pair_chunks(K))};
    *b = {nullptr, (uint8_t*)scratch + up256(a->bytes()), N, BN, int((N + BN - 1) / BN), a->chunks};
}

size_t dense_pair_workspace(int64_t M, int64_t N, int64_t K) {
    ScaleTiles a, b;
    dense_pair_tiles(M, N, K, nullptr, &a, &b);
    return size_t(up256(a.bytes()) + up256(b.bytes()));
}

namespace {

// Sizes and output of product q with tiles of bn columns; false when there are
// too many tiles.
bool set_problem(PairArgs& a, int q, const DenseArgs& d, int bn, bool early) {
    PairProblem& p = a.p[q];
    const bool gate = d.epi == kEpiGate;
    p.M = d.M;
    p.N = gate ? d.N / 2 : d.N;
    p.tiles_m = int((d.M + 255) / 256);
    p.bn = bn;
    const int64_t w = gate ? bn / 2 : bn, tn = (p.N + w - 1) / w;
    p.nks = int((d.K + (d.mx4 ? 255 : 63)) / (d.mx4 ? 256 : 64));
    p.amn = d.a.k_step != 1;
    p.early_b = early;
    p.vec_out = d.N % (d.out_f32 ? 4 : 8) == 0 && (reinterpret_cast<uintptr_t>(d.out) & 15) == 0;
    p.out = d.out;
    if (p.tiles_m * tn > (int64_t(1) << 28)) return false;
    p.tiles_n = int(tn);
    a.tiles[q] = p.tiles_m * int(tn);
    return true;
}

cudaError_t bf16_maps(PairMaps& m, int q, const DenseArgs& d, const PairProblem& p) {
    cudaError_t e = encode_map(&m.a[q], bf16_spec(d.a, d.M, d.K, 128, 0));
    if (e != cudaSuccess) return e;
    if (d.epi != kEpiGate) return encode_map(&m.b[q], bf16_spec(d.b, d.N, d.K, uint32_t(p.bn / 2), 0));
    DenseOperand w = d.b;  // gate and up rows: every other row, or the two halves
    if (d.interleaved) w.row *= 2;
    return encode_map(&m.b[q], bf16_spec(w, p.N, d.K, uint32_t(p.bn / 2), d.interleaved ? d.b.row : p.N * d.b.row));
}

}  // namespace

cudaError_t launch_dense_pair(const DenseArgs& d, bool early, cudaStream_t st) {
    PairArgs a{};
    if (!set_problem(a, 0, d, pair_width((d.M + 255) / 256, d.N, d.mx4 != 0), early)) return cudaErrorInvalidValue;
    a.out_f32 = d.out_f32;
    a.interleaved = d.interleaved;
    a.bias = d.bias;
    a.gu = d.gu;
    a.dgu = d.dgu;
    a.sums = d.sums;
    a.gate = d.gate;
    a.status = d.status;
    a.reset_status = d.reset_status;
    PairMaps maps = {};
    cudaError_t e;
    if (d.mx4) {
        if (!d.scratch) return cudaErrorInvalidValue;
        ScaleTiles t[2];
        dense_pair_tiles(d.M, d.N, d.K, d.scratch, &t[0], &t[1]);
        a.chunks = t[0].chunks;
        for (int i = 0; i < 2; ++i) {
            const MapSpec s = i ? mx4_spec(d.b.p, d.N, d.K, uint32_t(a.p[0].bn / 2)) : mx4_spec(d.a.p, d.M, d.K, 128);
            if ((e = encode_map(i ? &maps.b[0] : &maps.a[0], s)) != cudaSuccess) return e;
            MapSpec sc{};
            sc.p = t[i].out;
            sc.type = CU_TENSOR_MAP_DATA_TYPE_INT32;
            sc.dims[0] = 128;
            sc.dims[1] = uint64_t(t[i].bytes() / 512);
            sc.dims[2] = 1;
            sc.strides[0] = sc.strides[1] = 512;
            sc.box[0] = 128;
            sc.box[1] = uint32_t(2 * t[i].subs());  // a stage's two chunks
            sc.box[2] = 1;
            if ((e = encode_map(i ? &maps.b[1] : &maps.a[1], sc)) != cudaSuccess) return e;
        }
        return launch_one<true, false, false, kEpiStore>(maps, a, st);
    }
    if ((e = bf16_maps(maps, 0, d, a.p[0])) != cudaSuccess) return e;
    if (d.epi == kEpiGate) return launch_one<false, false, false, kEpiGate>(maps, a, st);
    if (d.epi == kEpiGateBwd) return launch_one<false, false, true, kEpiGateBwd>(maps, a, st);
    return launch_one<false, false, false, kEpiStore>(maps, a, st);
}

cudaError_t launch_dense_pairs(const DenseArgs* first, const DenseArgs* second, const DenseArgs* third, bool early3,
                               cudaStream_t st) {
    PairArgs a{};
    PairMaps maps = {};
    const DenseArgs* d[3] = {first, second, third};
    const int64_t m1 = second ? (second->M + 255) / 256 : 0, m2 = third ? (third->M + 255) / 256 : 0;
    const int width = pair_width(m1, second ? second->N : 0, false, m2, third ? third->N : 0);
    for (int q = 0; q < 3; ++q) {
        if (!d[q]) continue;
        const int bn = q == 0 ? pair_width((d[0]->M + 255) / 256, d[0]->N, false) : width;
        if (!set_problem(a, q, *d[q], bn, q == 2 ? early3 : true)) return cudaErrorInvalidValue;
        const cudaError_t e = bf16_maps(maps, q, *d[q], a.p[q]);
        if (e != cudaSuccess) return e;
        a.status = d[q]->status;
    }
    const int D = a.tiles[0], W = a.tiles[1] + a.tiles[2], pairs = sm_count() / 2;
    const int short_of = D && W && D + W > pairs && D % pairs ? pairs - D % pairs : 0;  // pairs with one fewer long tile
    if (short_of) {
        const PairProblem& s = second ? a.p[1] : a.p[2];
        const int64_t head = int64_t(a.p[0].nks) * (a.p[0].bn + 256) / (int64_t(s.nks) * (s.bn + 256));
        const int64_t most = (W + short_of - 1) / short_of;
        a.head = int(head < most ? head : most);
    }
    return launch_one<false, true, true, kEpiStore>(maps, a, st);
}

}  // namespace qmoe
