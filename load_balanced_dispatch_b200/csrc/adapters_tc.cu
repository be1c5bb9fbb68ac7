// adapters_tc.cu -- the router projection with a low-rank adapter per request on the tensor cores
// (bf16 activations). The operator is described in adapters.cu.
//
// Forward. Rows are grouped by adapter (adapters.cu, AdapterPlan), so that the 256 rows of a tile share
// one A_a; a tile's B operand is [W0; W1; W2; A_a], where W0 + W1 + W2 = W_r in three bf16 parts (every
// product exact, fp32 accumulation), and x is read once for the projection and the adapter together:
//   router_adapters_tc_kernel  one persistent CTA per SM, 384 threads:
//     warps 0,2,3 TMA, 64 columns a stage: warp 0 the B operand and the 32-row slabs of x whose rows follow
//                 one another, warps 2 and 3 the other slabs, four rows a gather
//     warp 1      tcgen05.mma, M = 128 twice (the two halves of the tile share the B operand)
//     warps 4-11  drain: a thread owns a row; every kDrain K blocks the accumulators are added into fp32
//                 registers with round-to-nearest adds (the tensor core's own adds truncate, so a long run
//                 in TMEM would drift); then the epilogue has s B_a u formed and stores logits and u.
// The K blocks of all tiles form one line that is cut into equal runs, one per CTA, whatever the groups'
// sizes are. A tile that a cut divides is finished by the last of its CTAs to arrive: each writes its
// partial sums and takes a ticket, nobody waits, and the sums are added in CTA order (the same bits
// whoever comes last).
#include "tc_ptx.cuh"

namespace moe {

namespace atc {
constexpr int BM = 256, BK = 64, kThreads = 384, kDrain = 4;
constexpr int A_BYTES = BM * BK * 2;
}  // namespace atc

// CTAs that share a line of `units` x nkb K blocks: every SM where there are units enough; else a whole number of
// CTAs per unit, each with at least kLeastRun K blocks (shorter runs spend their time on the partial sums).
constexpr int kLeastRun = 16;
__device__ __forceinline__ int64_t line_ctas(int64_t units, int nkb) {
    if (units >= (int64_t)gridDim.x || units == 0) return gridDim.x;
    int64_t f = gridDim.x / units;
    if (f > nkb / kLeastRun) f = nkb / kLeastRun;
    return units * (f < 1 ? 1 : f);
}

struct AtcShared {
    uint64_t full[4], empty[4], tfull, tempty, bfull;
    uint32_t tmem_base;
    int abort_flag;
    int last;
};

template <int NP, int RP>
struct AtcTile {
    static constexpr bool FUSED = 3 * NP + RP <= 256;
    static constexpr int ACOLS = FUSED ? 3 * NP + RP : NP + RP;  // accumulator columns of a half tile
    static constexpr int B_BYTES = (3 * NP + RP) * 128;
    static constexpr int STAGE = atc::A_BYTES + B_BYTES;
    static constexpr int STAGES = STAGE <= 65536 ? 3 : 2;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + (size_t)NP * 128 + 8 * 32 * 17 * 4 + sizeof(AtcShared);
    // three bf16 parts of s u, two values a column: over accumulators that have been read, or behind both halves'
    static constexpr int UCOL = FUSED ? NP : 2 * ACOLS, USTEP = FUSED ? ACOLS : 3 * RP / 2;
    static constexpr uint32_t TCOLS = FUSED && 2 * ACOLS <= 256 ? 256 : 512;
    static_assert(FUSED ? NP + 3 * RP / 2 <= ACOLS : 2 * ACOLS + 2 * USTEP <= 512, "the parts of u fit");
    static_assert(2 * ACOLS <= 512, "both halves' accumulators fit the TMEM");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// v = p[0] + p[1] + p[2], each bf16
__device__ __forceinline__ void split3(float v, __nv_bfloat16 (&p)[3]) {
    p[0] = __float2bfloat16_rn(v);
    const float r1 = v - __bfloat162float(p[0]);
    p[1] = __float2bfloat16_rn(r1);
    p[2] = __float2bfloat16_rn(r1 - __bfloat162float(p[1]));
}

// tile::gather4: four rows of 64 columns (the map's box is one row high)
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int r0, int r1,
                                            int r2, int r3) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
        : "memory");
}

template <int NP, int RP>
__global__ void __launch_bounds__(atc::kThreads, 1)
router_adapters_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                          const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                          const __nv_bfloat16* __restrict__ bmat, const float* __restrict__ scale, int d, int n, int r,
                          int na, int nct, AdapterPlan plan, float* __restrict__ part, int32_t* __restrict__ tickets,
                          float* __restrict__ logits, float* __restrict__ hidden) {
    using namespace atc;
    using T = AtcTile<NP, RP>;
    constexpr int STAGES = T::STAGES, ACOLS = T::ACOLS;
    constexpr uint32_t TCOLS = T::TCOLS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sB = smem + STAGES * T::STAGE;                         // B_a: [NP] rows of 128 bytes, swizzled
    float* stgs = reinterpret_cast<float*>(sB + NP * 128);          // 8 warps x [32][17]
    AtcShared* sh = reinterpret_cast<AtcShared*>(stgs + 8 * 32 * 17);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nkb = (d + BK - 1) / BK;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) { ptx::mbar_init(&sh->full[s], 3); ptx::mbar_init(&sh->empty[s], 1); }
        ptx::mbar_init(&sh->tfull, 1);
        ptx::mbar_init(&sh->tempty, 256);
        ptx::mbar_init(&sh->bfull, 1);
        sh->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&map_x);
        ptx::prefetch_tensormap(&map_g);
        ptx::prefetch_tensormap(&map_w);
        ptx::prefetch_tensormap(&map_a);
    }
    if (warp == 1) ptx::tmem_alloc(&sh->tmem_base, TCOLS);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    pdl_trigger();
    pdl_wait();  // the plan and the parts of W_r come from the launch before
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort_flag = &sh->abort_flag;

    const int groups = na + 1;
    const int64_t total = (int64_t)plan.tstart[groups] * nct * nkb;
    const int64_t ctas = line_ctas(total / nkb, nkb);
    const int64_t c = blockIdx.x;
    const int64_t lo = c < ctas ? c * total / ctas : total, hi = c < ctas ? (c + 1) * total / ctas : total;

    // unit -> tile and column tile, group, first grouped position, rows
    auto rows_of = [&](int64_t unit, int& ct, int& g, int& p0) -> int {
        const int tile = (int)(unit / nct);
        ct = (int)(unit % nct);
        g = group_at(plan.tstart, groups, tile);
        p0 = plan.goff[g] + BM * (tile - plan.tstart[g]);
        const int cnt = plan.goff[g] + plan.gcnt[g] - p0;
        return cnt < BM ? cnt : BM;
    };

    // 384 x 168 registers at launch = 128 x 72 + 256 x 216: the drain keeps a row's sums in registers
    const uint32_t leader = lane == 0 ? 1u : 0u;
    if (warp < 4) {
        ptx::regs_less<72>();
        if (warp != 1) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t pos = lo; ok && pos < hi;) {
                const int64_t unit = pos / nkb;
                const int kb0 = (int)(pos - unit * nkb);
                const int kb1 = (int)min((int64_t)nkb, kb0 + (hi - pos));
                int ct, g, p0;
                const int cnt = rows_of(unit, ct, g, p0);
                const bool ad = g < na;
                // lane s < 8 looks at slab s, the tile's rows 32 s .. 32 s + 31: one box if they follow one another
                const int left = cnt - 32 * (lane & 7);
                const int first = left > 0 ? plan.perm[p0 + 32 * (lane & 7)] : 0;
                const bool run = left > 0 && plan.perm[p0 + 32 * (lane & 7) + min(left, 32) - 1] - first == min(left, 32) - 1;
                const uint32_t boxes = __ballot_sync(0xffffffffu, run) & 0xffu;
                const uint32_t gathers = __ballot_sync(0xffffffffu, left > 0 && !run) & 0xffu;
                // warps 2 and 3: lane q gathers four rows of slab 4 (warp - 2) + q / 8
                const int slab = 4 * (warp & 1) + (lane >> 3), quad = 32 * slab + 4 * (lane & 7);
                const bool gather = warp >= 2 && (gathers >> slab & 1u) && quad < cnt;
                int rid[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) rid[q] = gather ? plan.perm[p0 + min(quad + q, cnt - 1)] : 0;
                // each of the three warps announces its own bytes, also none: a warp that a stage did not wait for
                // could fall a whole ring behind and then wait for a phase that has passed
                const uint32_t bytes = warp == 0 ? 3 * NP * 128 + (ad ? RP * 128 : 0) + __popc(boxes) * 4096
                                                 : __popc(__ballot_sync(0xffffffffu, gather)) * 512;
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag));
                    if (!ok) break;
                    uint8_t* st = smem + stage * T::STAGE;
                    uint8_t* sb = st + A_BYTES;
                    uint64_t* bar = &sh->full[stage];
                    if (lane == 0) ptx::mbar_expect_tx(bar, bytes);
                    __syncwarp();
                    if (warp == 0) {
                        // B rows: fused [W0 W1 W2 A], else [W0 A W1 W2]
                        if (lane >= 8 && lane < 11) {
                            const int p = lane - 8;
                            const int row = p * NP + (!T::FUSED && p > 0 ? RP : 0);
                            ptx::tma_load_3d(sb + row * 128, &map_w, bar, kb * BK, ct * NP, p);
                        }
                        if (lane == 11 && ad)
                            ptx::tma_load_3d(sb + (T::FUSED ? 3 * NP : NP) * 128, &map_a, bar, kb * BK, 0, g);
                        if (lane < 8 && run) ptx::tma_load_2d(st + lane * 4096, &map_x, bar, kb * BK, first);
                    } else if (gather) {
                        tma_gather4(st + quad * 128, &map_g, bar, kb * BK, rid[0], rid[1], rid[2], rid[3]);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                pos += kb1 - kb0;
            }
        } else {
            int stage = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            for (int64_t pos = lo; ok && pos < hi;) {
                const int64_t unit = pos / nkb;
                const int kb0 = (int)(pos - unit * nkb);
                const int kb1 = (int)min((int64_t)nkb, kb0 + (hi - pos));
                int ct, g, p0;
                const int cnt = rows_of(unit, ct, g, p0);
                const int halves = cnt > 128 ? 2 : 1, wide = g < na ? RP : 0;
                const uint32_t idesc = ptx::idesc_bf16_f32(128, (T::FUSED ? 3 * NP : NP) + wide);
                const uint32_t idesc_w = ptx::idesc_bf16_f32(128, NP);
                for (int kb = kb0; kb < kb1; ++kb) {
                    const int in = (kb - kb0) % kDrain;
                    if (in == 0) {
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->tempty, tphase ^ 1u, abort_flag));
                        if (!ok) break;
                    }
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->full[stage], phase, abort_flag));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t sa = ptx::smem_u32(smem + stage * T::STAGE);
                    const uint64_t bdesc = ptx::sw128_kmajor_desc(sa + A_BYTES);
                    for (int h = 0; h < halves; ++h) {
                        const uint64_t adesc = ptx::sw128_kmajor_desc(sa + h * 16384);
                        const uint32_t acc = tmem + (uint32_t)(h * ACOLS);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            ptx::umma_bf16_if(leader, acc, adesc + 2 * kk, bdesc + 2 * kk, idesc, (in != 0 || kk != 0) ? 1u : 0u);
                        if (!T::FUSED) {
#pragma unroll
                            for (int p = 1; p < 3; ++p) {
                                const uint64_t wdesc = ptx::sw128_kmajor_desc(sa + A_BYTES + (p * NP + RP) * 128);
#pragma unroll
                                for (int kk = 0; kk < BK / 16; ++kk)
                                    ptx::umma_bf16_if(leader, acc, adesc + 2 * kk, wdesc + 2 * kk, idesc_w, 1u);
                            }
                        }
                    }
                    ptx::umma_commit_if(leader, &sh->empty[stage]);
                    if (in == kDrain - 1 || kb == kb1 - 1) { ptx::umma_commit_if(leader, &sh->tfull); tphase ^= 1u; }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                pos += kb1 - kb0;
            }
        }
    } else {
        ptx::regs_more<216>();
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int row = half * 128 + quad * 32 + lane;  // of the tile
        const int et = tid - 128;                       // 0 .. 255
        float* stg = stgs + (warp - 4) * 32 * 17;
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * ACOLS);
        uint32_t tphase = 0, bphase = 0;
        bool ok = true;
        for (int64_t pos = lo; pos < hi;) {
            const int64_t unit = pos / nkb;
            const int kb0 = (int)(pos - unit * nkb);
            const int kb1 = (int)min((int64_t)nkb, kb0 + (hi - pos));
            int ct, g, p0;
            const int cnt = rows_of(unit, ct, g, p0);
            const bool ad = g < na, mine = half * 128 < cnt;
            float acc[NP], u[RP];
#pragma unroll
            for (int j = 0; j < NP; ++j) acc[j] = 0.f;
#pragma unroll
            for (int j = 0; j < RP; ++j) u[j] = 0.f;
            for (int kb = kb0; kb < kb1; kb += kDrain) {
                // after a give-up every warp still walks its loops: the barriers below count them all
                if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->tfull, tphase, abort_flag));
                tphase ^= 1u;
                if (!ok) continue;
                ptx::tc_fence_after();
                if (mine) {
#pragma unroll
                    for (int q = 0; q < NP / 16; ++q) {
                        uint32_t v[T::FUSED ? 3 : 1][16];
#pragma unroll
                        for (int p = 0; p < (T::FUSED ? 3 : 1); ++p) ptx::tmem_ld16_issue(trow + (uint32_t)(p * NP + q * 16), v[p]);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float b = __uint_as_float(v[0][j]);
                            if constexpr (T::FUSED)
                                b = __fadd_rn(__fadd_rn(__uint_as_float(v[2][j]), __uint_as_float(v[1][j])), b);
                            acc[q * 16 + j] = __fadd_rn(acc[q * 16 + j], b);
                        }
                    }
                    if (ad) {
#pragma unroll
                        for (int q = 0; q < RP / 16; ++q) {
                            uint32_t v[16];
                            ptx::tmem_ld16_issue(trow + (uint32_t)((T::FUSED ? 3 * NP : NP) + q * 16), v);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[q * 16 + j] = __fadd_rn(u[q * 16 + j], __uint_as_float(v[j]));
                        }
                    }
                }
                ptx::tc_fence_before();
                if (kb + kDrain < kb1) ptx::mbar_arrive(&sh->tempty);  // the last arrival comes below
            }
            bool finish = true;
            if (kb0 != 0 || kb1 != nkb) {
                // a part of the unit: leave the sums, and finish it if every other part is there already
                // [column / 4][row][4]: 16-byte accesses, a warp's rows beside one another
                float4* mp = reinterpret_cast<float4*>(part) + (2 * c + (kb0 == 0 ? 1 : 0)) * (int64_t)(NP + RP) / 4 * BM + row;
                if (ok && row < cnt) {
#pragma unroll
                    for (int j = 0; j < NP; j += 4) __stcg(mp + (int64_t)(j / 4) * BM, make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
                    if (ad) {
#pragma unroll
                        for (int j = 0; j < RP; j += 4)
                            __stcg(mp + (int64_t)((NP + j) / 4) * BM, make_float4(u[j], u[j + 1], u[j + 2], u[j + 3]));
                    }
                }
                __threadfence();
                ptx::named_barrier(1, 256);
                const int64_t u0 = unit * nkb;
                const int64_t cf = ((u0 + 1) * ctas + total - 1) / total - 1, cl = ((u0 + nkb) * ctas + total - 1) / total - 1;
                if (et == 0) sh->last = atomicAdd(tickets + unit, 1) == (int)(cl - cf);
                ptx::named_barrier(1, 256);
                finish = sh->last != 0;
                if (finish) {
                    __threadfence();
#pragma unroll
                    for (int j = 0; j < NP; ++j) acc[j] = 0.f;
#pragma unroll
                    for (int j = 0; j < RP; ++j) u[j] = 0.f;
                    if (row < cnt) {
                        for (int64_t cc = cf; cc <= cl; ++cc) {
                            const int64_t at = cc * total / ctas;  // where the CTA's run begins
                            const float4* op = reinterpret_cast<const float4*>(part) + (2 * cc + (at <= u0 ? 1 : 0)) * (int64_t)(NP + RP) / 4 * BM + row;
#pragma unroll
                            for (int j = 0; j < NP; j += 4) {
                                const float4 t = __ldcg(op + (int64_t)(j / 4) * BM);
                                acc[j] = __fadd_rn(acc[j], t.x); acc[j + 1] = __fadd_rn(acc[j + 1], t.y);
                                acc[j + 2] = __fadd_rn(acc[j + 2], t.z); acc[j + 3] = __fadd_rn(acc[j + 3], t.w);
                            }
                            if (ad) {
#pragma unroll
                                for (int j = 0; j < RP; j += 4) {
                                    const float4 t = __ldcg(op + (int64_t)((NP + j) / 4) * BM);
                                    u[j] = __fadd_rn(u[j], t.x); u[j + 1] = __fadd_rn(u[j + 1], t.y);
                                    u[j + 2] = __fadd_rn(u[j + 2], t.z); u[j + 3] = __fadd_rn(u[j + 3], t.w);
                                }
                            }
                        }
                    }
                }
            }
            if (finish && ad) {  // the same for all eight warps
                // s B_a u by the tensor core: s u in three bf16 parts that add up to it, in tensor memory, and B_a
                // (exact) in shared memory. Against products by FMA: 41 for 54 us (8191 rows of 768, n 128, rank 8), 148
                // for 155 us (65536 rows of 4096, n 64, rank 16)
                if (ok) {
                    const float s = scale[g];
                    const uint32_t ut = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(T::UCOL + half * T::USTEP);
#pragma unroll
                    for (int q = 0; q < RP; q += 32) {
                        uint32_t v[3][16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            __nv_bfloat16 a0[3], a1[3];
                            split3(s * u[q + j], a0);
                            split3(s * u[q + j + 1], a1);
#pragma unroll
                            for (int p = 0; p < 3; ++p) {
                                const __nv_bfloat162 two(a0[p], a1[p]);
                                v[p][j / 2] = *reinterpret_cast<const uint32_t*>(&two);
                            }
                        }
#pragma unroll
                        for (int p = 0; p < 3; ++p) ptx::tmem_st16_issue(ut + (uint32_t)(p * (RP / 2) + q / 2), v[p]);
                    }
                    ptx::tmem_wait_st();
                }
                for (int i = et; i < NP * RP / 8; i += 256) {  // 16-byte piece i % (RP / 8) of row i / (RP / 8)
                    const int e = i / (RP / 8), c8 = i % (RP / 8), col = ct * NP + e;
                    const __nv_bfloat16* src = bmat + ((int64_t)g * n + col) * r + 8 * c8;
                    uint32_t v[4] = {0u, 0u, 0u, 0u};
                    if (col < n) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (8 * c8 + j < r) v[j / 2] |= (uint32_t)__bfloat16_as_ushort(src[j]) << (16 * (j & 1));
                    }
                    *reinterpret_cast<uint4*>(sB + e * 128 + ((c8 ^ (e & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
                }
                ptx::fence_proxy_async_shared();
                ptx::tc_fence_before();
                ptx::named_barrier(1, 256);
                if (et == 0) {
                    ptx::tc_fence_after();
                    const uint32_t idesc = ptx::idesc_bf16_f32(128, NP);
                    const uint64_t bdesc = ptx::sw128_kmajor_desc(ptx::smem_u32(sB));
                    for (int h = 0; h < (cnt > 128 ? 2 : 1); ++h)
                        for (int p = 2; p >= 0; --p)  // the small parts first
                            for (int k = 0; 16 * k < r; ++k)
                                ptx::umma_bf16_ts(tmem + (uint32_t)(h * ACOLS), tmem + (uint32_t)(T::UCOL + h * T::USTEP + p * (RP / 2) + 8 * k),
                                                  bdesc + 2 * k, idesc, (p != 2 || k != 0) ? 1u : 0u);
                    ptx::umma_commit(&sh->bfull);
                }
                __syncwarp();
                if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->bfull, bphase, abort_flag));
                bphase ^= 1u;
                ptx::tc_fence_after();
                if (ok && mine) {
#pragma unroll
                    for (int q = 0; q < NP / 16; ++q) {
                        uint32_t v[16];
                        ptx::tmem_ld16_issue(trow + (uint32_t)(q * 16), v);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[q * 16 + j] = __fadd_rn(acc[q * 16 + j], __uint_as_float(v[j]));
                    }
                }
                ptx::tc_fence_before();
            }
            if (ok) ptx::mbar_arrive(&sh->tempty);  // the accumulators are free for the next unit
            if (finish) {
                // 16 columns at a time through the warp's staging rows: stores of 64-byte pieces
                if (ok && half * 128 + quad * 32 < cnt) {  // the same for the warp
                    const int32_t out = row < cnt ? plan.perm[p0 + row] : -1;
                    float* mine = stg + lane * 17;
                    int32_t to[16];  // the row of each of this lane's pieces
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i] = __shfl_sync(0xffffffffu, out, 2 * i + (lane >> 4));
                    const float* from = stg + (lane >> 4) * 17 + (lane & 15);
                    auto store16 = [&](float* dst, int width, int col) {
                        const int cc = col + (lane & 15);
                        __syncwarp();
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = from[i * 34];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (to[i] >= 0 && cc < width) dst[(int64_t)to[i] * width + cc] = v[i];
                        __syncwarp();
                    };
                    if (hidden && ct == 0) {
#pragma unroll
                        for (int q = 0; q < RP; q += 16) {
                            if (q < r) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) mine[j] = u[q + j];
                                store16(hidden, r, q);
                            }
                        }
                    }
#pragma unroll
                    for (int e0 = 0; e0 < NP; e0 += 16) {
                        if (ct * NP + e0 < n) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) mine[j] = acc[e0 + j];
                            store16(logits, n, ct * NP + e0);
                        }
                    }
                }
            }
            pos += kb1 - kb0;
        }
    }
    ptx::settle_after_abort(abort_flag);
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TCOLS);
    }
}

// ---- host side
// Column tile of the logits: all n in one tile where the accumulators fit, else equal tiles; 64 columns at most where
// that gives more CTAs work (8191 rows of 768 columns, n 128: 34 us with one tile of 128, 20 with two of 64).
static void atc_tile(int64_t m, int n, int r, int& np, int& rp, int& nct) {
    rp = r <= 32 ? 32 : 64;
    const int most = rp == 32 && 2 * (m / atc::BM + 1) > kNumSMs ? 128 : 64;
    nct = (n + most - 1) / most;
    np = ((n + nct - 1) / nct + 31) / 32 * 32;
}

struct AtcWs {
    AdapterPlan plan;
    __nv_bfloat16* wsplit;  // [3, n, d]
    float* part;            // [2 kNumSMs][NP + RP][256]
    int32_t* tickets;       // one per unit
};

static int64_t atc_tiles(int64_t m, int na) { return m / atc::BM + na + 1; }

static size_t atc_layout(int64_t m, int d, int n, int r, int na, AtcWs* w, char* base) {
    int np, rp, nct;
    atc_tile(m, n, r, np, rp, nct);
    size_t off = 0;
    auto take = [&](size_t bytes) { char* p = base + off; off += (bytes + 255) & ~size_t(255); return p; };
    off = adapter_plan_layout(m, na, w ? &w->plan : nullptr, base);
    char* p;
    p = take((size_t)3 * n * d * 2);                                 if (w) w->wsplit = (__nv_bfloat16*)p;
    p = take((size_t)2 * kNumSMs * (np + rp) * atc::BM * 4);          if (w) w->part = (float*)p;
    p = take(4 * (size_t)(atc_tiles(m, na) * nct));                   if (w) w->tickets = (int32_t*)p;
    return off;
}

template <int NP, int RP>
static cudaError_t launch_atc(const CUtensorMap& mx, const CUtensorMap& mg, const CUtensorMap& mw,
                              const CUtensorMap& ma, const __nv_bfloat16* b, const float* scale, int d, int n, int r,
                              int na, int nct, const AtcWs& w, float* logits, float* hidden, cudaStream_t stream) {
    constexpr size_t smem = AtcTile<NP, RP>::SMEM;
    const cudaError_t e = need_smem<router_adapters_tc_kernel<NP, RP>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(router_adapters_tc_kernel<NP, RP>, dim3(kNumSMs), dim3(atc::kThreads), smem, stream, mx, mg, mw,
                      ma, b, scale, d, n, r, na, nct, w.plan, w.part, w.tickets, logits, hidden);
}

static cudaError_t launch_router_adapters_tc(const __nv_bfloat16* x, const float* w_r, const __nv_bfloat16* a,
                                             const __nv_bfloat16* b, const int32_t* idx, const float* scale, int64_t m,
                                             int d, int n, int r, int na, float* logits, float* hidden, void* workspace,
                                             cudaStream_t stream) {
    int np, rp, nct;
    atc_tile(m, n, r, np, rp, nct);
    AtcWs w;
    atc_layout(m, d, n, r, na, &w, static_cast<char*>(workspace));
    PrepExtra extra = {};
    extra.w_r = w_r; extra.d = d; extra.n = n; extra.wparts = w.wsplit;
    const cudaError_t e = launch_adapter_prep(idx, m, na, w.plan, w.tickets, atc_tiles(m, na) * nct, extra, stream);
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mg, mw, ma;
    if (!map_2d(&mx, x, (uint64_t)m, (uint64_t)d, 32) || !map_2d(&mg, x, (uint64_t)m, (uint64_t)d, 1) ||
        !map_3d(&mw, w.wsplit, 3, (uint64_t)n, (uint64_t)d, (uint32_t)np) ||
        !map_3d(&ma, a, (uint64_t)na, (uint64_t)r, (uint64_t)d, (uint32_t)rp))
        return cudaErrorInvalidValue;
#define MOE_ATC(NP, RP) return launch_atc<NP, RP>(mx, mg, mw, ma, b, scale, d, n, r, na, nct, w, logits, hidden, stream)
    if (rp == 32) {
        if (np == 32) MOE_ATC(32, 32);
        if (np == 64) MOE_ATC(64, 32);
        if (np == 96) MOE_ATC(96, 32);
        MOE_ATC(128, 32);
    }
    if (np == 32) MOE_ATC(32, 64);
    MOE_ATC(64, 64);
#undef MOE_ATC
}

}  // namespace moe
