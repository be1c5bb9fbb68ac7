// adapters_grad_tc.cu -- backward of the router projection with adapters on the tensor cores (bf16
// activations). The operator is described in adapters.cu; rows are in the grouped order of AdapterPlan.
//
//   adapters_split_kernel     per row: du = s B_a^T dh, and dh and du as 16-bit parts that add up to the fp32
//                             value (bf16 for the weight gradients, scaled fp16 and bf16 for dx); dB on the way,
//                             each CTA's sums over its run of rows to a slot of its own
//   adapters_dx_tc_kernel     dx = dh W_r^T + du A_a: the parts of dh and du of a row tile stay in shared
//                             memory while the parts of W_r and A_a stream past, columns of d at a time
//   rows_contract_tc_kernel   dA_a = du^T x and dW_r = x^T dh: a contraction over rows, x read once per 64
//                             columns of the other operand
//   adapters_fold_kernel      dB from the slots, zeros for adapters without rows
//
// All sums are right to fp32. For the weight gradients x (exact in bf16) meets three bf16 parts. For dx both sides
// are fp32: dh and W_r are multiplied by powers of two (one a row of dh, one a row of W_r), so that two fp16 parts
// hold 22 bits of each value, and three of their four products are formed (the fourth is below 2^-22); du A_a, du in
// three bf16 parts, is scaled alike and added to the same sums; the drain takes the powers out again. Two bf16 parts a
// side without scales have 16 bits, which shows in dx where W_r's rows have much in common (the gradient of a
// softmax adds up to zero, so that cancels). dx of 65536 rows, d 4096, n 64, rank 16: 131 us with two bf16 parts,
// 142 us so, 205 us with three bf16 parts and six products.
#include "tc_ptx.cuh"

namespace moe {

// K rows in memory order, MN contiguous: boxes of 64 MN columns x K rows under the 128-byte swizzle. The
// next 64 columns are `lbo` bytes on, the next eight rows 1024.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lbo >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;  // operand A / B is MN-major

namespace asp {
constexpr int kThreads = 256, kGrid = 2 * kNumSMs, kRows = adp::kPad;
}

// What the contractions and dx read, [rows in the grouped order]. Null pointers: not wanted.
struct SplitOut {
    __nv_bfloat16 *dhp;  // [3, m_pad, nk] dh in three bf16 parts (dW_r)
    __nv_bfloat16 *dup;  // [m_pad, 128 or 192] du in three bf16 parts beside one another (dA)
    __half* dhs;         // [2, m_pad, nk] dh times 2^k of its row in two fp16 parts (dx)
    __nv_bfloat16 *dus;  // as dup, du times 2^k (dx)
    float* rinv;         // [m_pad] 2^-k
};

// CTA c takes the row blocks (kRows grouped positions) c nb / ctas .. (c + 1) nb / ctas - 1. A group's
// part of dB in CTA c goes to slot c + g: unique, since each next slot advances the CTA or the group.
// LPR lanes load a row of dh, NQ 16-byte pieces each. Thread (te, tj) owns dB[NE te + a][NJ tj + b]; du has four
// threads a row, each a quarter of the padded rank.
template <int NE, int NJ, int RP>
__global__ void __launch_bounds__(asp::kThreads)
adapters_split_kernel(const float* __restrict__ dh, const float* __restrict__ hidden,
                      const __nv_bfloat16* __restrict__ bmat, const float* __restrict__ scale, int n, int r, int na,
                      AdapterPlan plan, int nk, int64_t mp, SplitOut out, float* __restrict__ slots) {
    using namespace asp;
    constexpr int NP = NE * 32, HS = NP + 4, US = RP + 4;  // rows 4 words apart from a multiple of 32: no bank conflicts
    constexpr int LPR = NP == 64 ? 16 : 32, NQ = NP / (4 * LPR), JT = RP / 4, PC = RP == 32 ? 128 : 192;
    constexpr int PASSES = kRows * LPR / kThreads;
    extern __shared__ float sm[];
    float* sh = sm;                 // [kRows][HS] dh
    float* su = sh + kRows * HS;    // [kRows][US] u
    float* sb = su + kRows * US;    // [RP][HS] B_a transposed; row j sits at (j % JT) * 4 + j / JT
    __shared__ float srow[kRows];   // 2^k of each row
    const int tid = threadIdx.x, te = tid >> 3, tj = tid & 7;
    const int lrow = tid / LPR, lcol = tid % LPR;
    pdl_trigger();
    pdl_wait();
    const int nb = plan.goff[na + 1] / kRows;
    const int ctas = min((int)gridDim.x, nb), c = (int)blockIdx.x;  // every CTA below `ctas` has a block
    const int b0 = c < ctas ? (int)((int64_t)c * nb / ctas) : 0, b1 = c < ctas ? (int)((int64_t)(c + 1) * nb / ctas) : 0;
    const bool vec = (n & 3) == 0, uvec = (r & 3) == 0;
    float acc[NE][NJ];
    int g = -1;
    auto flush = [&]() {
        if (g < 0 || g >= na) return;
        float* to = slots + ((int64_t)c + g) * n * r;
#pragma unroll
        for (int a = 0; a < NE; ++a)
#pragma unroll
            for (int b = 0; b < NJ; ++b) {
                const int e = NE * te + a, j = NJ * tj + b;
                if (e < n && j < r) to[e * r + j] = acc[a][b];
            }
    };
    for (int blk = b0; blk < b1; ++blk) {
        const int p0 = blk * kRows;
        int ng = g < 0 ? group_at(plan.goff, na + 1, p0) : g;
        while (plan.goff[ng + 1] <= p0) ++ng;
        __syncthreads();  // the block before is done with the tiles
        if (ng != g) {
            flush();
            g = ng;
#pragma unroll
            for (int a = 0; a < NE; ++a)
#pragma unroll
                for (int b = 0; b < NJ; ++b) acc[a][b] = 0.f;
            if (g < na)
                for (int i = tid; i < NP * RP; i += kThreads) {
                    const int e = i / RP, j = i % RP;
                    sb[((j % JT) * 4 + j / JT) * HS + e] = (e < n && j < r) ? __bfloat162float(bmat[((int64_t)g * n + e) * r + j]) : 0.f;
                }
        }
        // dh rows: registers -> shared memory, and their bf16 parts
        int32_t rows[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) rows[i] = plan.perm[p0 + lrow + kThreads / LPR * i];
        float4 v[PASSES][NQ];
#pragma unroll
        for (int i = 0; i < PASSES; ++i)
#pragma unroll
            for (int w = 0; w < NQ; ++w) {
                const int e = 4 * (lcol + LPR * w);
                v[i][w] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (rows[i] >= 0) {
                    const float* src = dh + (int64_t)rows[i] * n + e;
                    if (vec) {
                        if (e < n) v[i][w] = *reinterpret_cast<const float4*>(src);
                    } else {
                        if (e < n) v[i][w].x = src[0];
                        if (e + 1 < n) v[i][w].y = src[1];
                        if (e + 2 < n) v[i][w].z = src[2];
                        if (e + 3 < n) v[i][w].w = src[3];
                    }
                }
            }
        if (g < na) {
            for (int i = tid; i < kRows * (RP / 4); i += kThreads) {
                const int q = i / (RP / 4), j = 4 * (i % (RP / 4));
                const int32_t row = plan.perm[p0 + q];
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0 && j < r) {
                    const float* src = hidden + (int64_t)row * r + j;
                    if (uvec) {
                        t = *reinterpret_cast<const float4*>(src);
                    } else {
                        t.x = src[0];
                        if (j + 1 < r) t.y = src[1];
                        if (j + 2 < r) t.z = src[2];
                        if (j + 3 < r) t.w = src[3];
                    }
                }
                *reinterpret_cast<float4*>(su + q * US + j) = t;
            }
        }
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int q = lrow + kThreads / LPR * i;
            float up = 1.f;
            if (out.dhs) {  // the row's largest value sets its exponent
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < NQ; ++c)
                    top = fmaxf(fmaxf(fmaxf(top, fabsf(v[i][c].x)), fabsf(v[i][c].y)), fmaxf(fabsf(v[i][c].z), fabsf(v[i][c].w)));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int k = fit_exponent(top, kRowExponent);
                up = ldexpf(1.f, k);
                if (lcol == 0) { srow[q] = up; out.rinv[p0 + q] = ldexpf(1.f, -k); }
            }
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                const int e = 4 * (lcol + LPR * c);
                *reinterpret_cast<float4*>(sh + q * HS + e) = v[i][c];
                if (out.dhs && e < nk) {
                    __half p[4][2];
                    split2h(up * v[i][c].x, p[0]);
                    split2h(up * v[i][c].y, p[1]);
                    split2h(up * v[i][c].z, p[2]);
                    split2h(up * v[i][c].w, p[3]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const __half2 lo(p[0][k], p[1][k]), hi(p[2][k], p[3][k]);
                        *reinterpret_cast<uint2*>(out.dhs + ((int64_t)k * mp + p0 + q) * nk + e) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                }
                if (out.dhp && e < nk) {
                    __nv_bfloat16 p[4][3];
                    split3(v[i][c].x, p[0]);
                    split3(v[i][c].y, p[1]);
                    split3(v[i][c].z, p[2]);
                    split3(v[i][c].w, p[3]);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        const __nv_bfloat162 lo(p[0][k], p[1][k]), hi(p[2][k], p[3][k]);
                        *reinterpret_cast<uint2*>(out.dhp + ((int64_t)k * mp + p0 + q) * nk + e) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    }
                }
            }
        }
        if (g >= na) continue;
        __syncthreads();
        {   // du: row tid / 4, ranks (tid % 4) JT .. + JT - 1
            const int q = tid >> 2, part = tid & 3;
            float t[JT];
#pragma unroll
            for (int b = 0; b < JT; ++b) t[b] = 0.f;
            if (part * JT < r) {
                for (int e = 0; e < n; e += 4) {  // columns behind n are zero in both tiles
                    const float4 h = *reinterpret_cast<const float4*>(sh + q * HS + e);
#pragma unroll
                    for (int b = 0; b < JT; ++b) {
                        const float4 w = *reinterpret_cast<const float4*>(sb + (b * 4 + part) * HS + e);
                        t[b] = fmaf(h.x, w.x, fmaf(h.y, w.y, fmaf(h.z, w.z, fmaf(h.w, w.w, t[b]))));
                    }
                }
            }
            const float s = scale[g];
            auto store = [&](__nv_bfloat16* o, float up) {
#pragma unroll
                for (int b = 0; b < JT; b += 8) {
                    __nv_bfloat16 p[8][3];
#pragma unroll
                    for (int c = 0; c < 8; ++c) split3(s * t[b + c] * up, p[c]);
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        uint32_t u[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const __nv_bfloat162 two(p[2 * c][k], p[2 * c + 1][k]);
                            u[c] = *reinterpret_cast<const uint32_t*>(&two);
                        }
                        *reinterpret_cast<uint4*>(o + k * RP + b) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            };
            const int64_t at = (int64_t)(p0 + q) * PC + part * JT;
            // ranks behind r: dA's are not stored, dx's are multiplied up to whole 16
            if (part * JT < r) store(out.dup + at, 1.f);
            if (out.dus && part * JT < (r + 15) / 16 * 16) store(out.dus + at, srow[q]);
        }
        float part[NE][NJ];
#pragma unroll
        for (int a = 0; a < NE; ++a)
#pragma unroll
            for (int b = 0; b < NJ; ++b) part[a][b] = 0.f;
#pragma unroll 4
        for (int q = 0; q < kRows; ++q) {
            float hv[NE], uv[NJ];
#pragma unroll
            for (int a = 0; a < NE; a += 2) *reinterpret_cast<float2*>(hv + a) = *reinterpret_cast<const float2*>(sh + q * HS + NE * te + a);
#pragma unroll
            for (int b = 0; b < NJ; b += 2) *reinterpret_cast<float2*>(uv + b) = *reinterpret_cast<const float2*>(su + q * US + NJ * tj + b);
#pragma unroll
            for (int a = 0; a < NE; ++a)
#pragma unroll
                for (int b = 0; b < NJ; ++b) part[a][b] = fmaf(hv[a], uv[b], part[a][b]);
        }
#pragma unroll
        for (int a = 0; a < NE; ++a)
#pragma unroll
            for (int b = 0; b < NJ; ++b) acc[a][b] += part[a][b];
    }
    flush();
}

// db[g] = s_g * the group's slots, in CTA order; da[g] = 0 for a group without rows.
__global__ void __launch_bounds__(asp::kThreads)
adapters_fold_kernel(const float* __restrict__ slots, int n, int r, int d, int na, AdapterPlan plan,
                     const float* __restrict__ scale, float* __restrict__ db, float* __restrict__ da) {
    using namespace asp;
    pdl_trigger();
    pdl_wait();
    const int g = blockIdx.y;
    const int per = n * r;
    const int nb = plan.goff[na + 1] / kRows, b0 = plan.goff[g] / kRows, b1 = plan.goff[g + 1] / kRows;
    const int i0 = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
    if (b1 == b0) {
        for (int i = i0; i < per; i += step) db[(int64_t)g * per + i] = 0.f;
        for (int64_t i = i0; i < (int64_t)r * d; i += step) da[(int64_t)g * r * d + i] = 0.f;
        return;
    }
    // the CTA of block b: the last c with c nb / ctas <= b
    const int ctas = min(kGrid, nb);
    const int cf = (int)((((int64_t)b0 + 1) * ctas + nb - 1) / nb) - 1, cl = (int)(((int64_t)b1 * ctas + nb - 1) / nb) - 1;
    for (int i = i0; i < per; i += step) {
        float t = 0.f;
#pragma unroll 8
        for (int c = cf; c <= cl; ++c) t += slots[((int64_t)c + g) * per + i];
        db[(int64_t)g * per + i] = scale[g] * t;
    }
}

// ---------------------------------------------------------------- dx
namespace adx {
constexpr int kThreads = 384, kMaxSlots = 4;
}

struct AdxShared {
    uint64_t full[adx::kMaxSlots], empty[adx::kMaxSlots], afull, aempty, tfull[2], tempty[2];
    uint32_t tmem_base;
    int abort_flag;
};

// ND: columns of d at a time; NC: 64-column chunks of dh; RP: padded rank. N is 256 where the two accumulators and the
// ring allow it: 128 columns for 256 rows at a time measured 152 us against 132 us (65536 rows, d 4096, n 64, rank 16,
// two bf16 parts). Both the MMAs and the drain count: 13 more MMAs a unit cost 74 us there, and loads of the column
// factors inside the drain's loop 36 us.
template <int ND, int NC, int RP>
struct AdxTile {
    static constexpr int DH_BYTES = 2 * NC * 16384;             // [plane][chunk] of 128 rows of 128 bytes
    static constexpr int DU_ALL = RP == 32 ? 2 : 3;             // du's parts: [p0 | p1], [p2 | -] for rank 32, else a chunk each
    static constexpr bool STREAM = NC == 4;                     // p2 comes through the ring, behind A_a
    static constexpr int DU_CHUNKS = STREAM ? DU_ALL - 1 : DU_ALL;
    static constexpr int A_BYTES = DH_BYTES + DU_CHUNKS * 16384;
    static constexpr int SLOT = ND * 128;                       // 64 columns of a part of W_r, or A_a
    static constexpr int OUT_BYTES = 8 * 32 * 64 * 2;
    static constexpr int ROOM = 227 * 1024 - 1024 - A_BYTES - OUT_BYTES - (int)sizeof(AdxShared);
    static constexpr int SLOTS = ROOM / SLOT < adx::kMaxSlots ? ROOM / SLOT : adx::kMaxSlots;
    static constexpr size_t SMEM = 1024 + A_BYTES + SLOTS * SLOT + OUT_BYTES + sizeof(AdxShared);
    static_assert(SLOTS >= 2, "a slot is filled while another is read");
    static_assert(2 * ND <= 512, "two accumulators fit the TMEM");
    static_assert(ND / 64 * RP * 128 <= SLOT && SLOT >= 16384, "A_a and a chunk of du fit a slot");
};

// The drain's products with powers of two, on values that are rounded already (exact).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&t);
}

// One unit = 128 grouped rows x ND columns of d; the units of a row tile follow one another, and the line of units is
// cut evenly over the CTAs.
//   warp 0 TMA, warp 1 MMA, warps 4-11 TMEM -> bf16 -> shared memory -> whole 128-byte pieces of dx rows
template <int ND, int NC, int RP>
__global__ void __launch_bounds__(adx::kThreads, 1)
adapters_dx_tc_kernel(const __grid_constant__ CUtensorMap map_dh, const __grid_constant__ CUtensorMap map_du,
                      const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, int d, int r,
                      int na, AdapterPlan plan, const float* __restrict__ rinv, const __nv_bfloat16* __restrict__ cinv,
                      __nv_bfloat16* __restrict__ dx) {
    using namespace adx;
    using T = AdxTile<ND, NC, RP>;
    constexpr int SLOTS = T::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sa = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* su = sa + T::DH_BYTES;
    uint8_t* ring = sa + T::A_BYTES;
    uint8_t* outs = ring + SLOTS * T::SLOT;
    AdxShared* sh = reinterpret_cast<AdxShared*>(outs + T::OUT_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < SLOTS; ++s) { ptx::mbar_init(&sh->full[s], 1); ptx::mbar_init(&sh->empty[s], 1); }
        ptx::mbar_init(&sh->afull, 1);
        ptx::mbar_init(&sh->aempty, 1);
        for (int b = 0; b < 2; ++b) { ptx::mbar_init(&sh->tfull[b], 1); ptx::mbar_init(&sh->tempty[b], 256); }
        sh->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&map_dh);
        ptx::prefetch_tensormap(&map_du);
        ptx::prefetch_tensormap(&map_w);
        ptx::prefetch_tensormap(&map_a);
    }
    if (warp == 1) ptx::tmem_alloc(&sh->tmem_base, 2 * ND);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    pdl_trigger();
    pdl_wait();
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort_flag = &sh->abort_flag;
    const int groups = na + 1, ndc = (d + ND - 1) / ND;
    const int64_t total = (int64_t)plan.tstart[groups] * 2 * ndc;
    const int64_t lo = blockIdx.x * total / gridDim.x, hi = (blockIdx.x + 1) * total / gridDim.x;

    // row tile -> group, first grouped position, rows (0: nothing to do)
    auto rows_of = [&](int64_t tile, int& g, int& p0) -> int {
        const int t = (int)(tile >> 1);
        g = group_at(plan.tstart, groups, t);
        p0 = plan.goff[g] + 256 * (t - plan.tstart[g]) + 128 * (int)(tile & 1);
        const int cnt = plan.goff[g] + plan.gcnt[g] - p0;
        return cnt < 0 ? 0 : min(cnt, 128);
    };

    const uint32_t leader = lane == 0 ? 1u : 0u;
    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, aphase = 0;
        int64_t held = -1;
        int g = 0, p0 = 0, cnt = 0;
        bool ok = true;
        for (int64_t u = lo; ok && u < hi; ++u) {
            const int64_t tile = u / ndc;
            const int d0 = (int)(u - tile * ndc) * ND;
            if (tile != held) {
                held = tile;
                cnt = rows_of(tile, g, p0);
                if (cnt > 0) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->aempty, aphase ^ 1u, abort_flag));
                    if (!ok) break;
                    aphase ^= 1u;
                    if (leader) ptx::mbar_expect_tx(&sh->afull, (uint32_t)(16384 * (2 * NC + (g < na ? T::DU_CHUNKS : 0))));
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int c = 0; c < NC; ++c)
                            ptx::tma_load_3d_if(leader, sa + (p * NC + c) * 16384, &map_dh, &sh->afull, 64 * c, p0, p);
                    if (g < na) {
#pragma unroll
                        for (int c = 0; c < T::DU_CHUNKS; ++c)
                            ptx::tma_load_2d_if(leader, su + c * 16384, &map_du, &sh->afull, 64 * c, p0);
                    }
                }
            }
            if (cnt == 0) continue;
            // slots in order: both parts of each chunk of W_r, then A_a, then (STREAM) the third part of du
            for (int c = 0; c < 2 * NC + (g < na ? (T::STREAM ? 2 : 1) : 0); ++c) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag));
                if (!ok) break;
                uint8_t* st = ring + stage * T::SLOT;
                if (leader) ptx::mbar_expect_tx(&sh->full[stage], c < 2 * NC ? ND * 128 : c == 2 * NC ? ND / 64 * RP * 128 : 16384);
                __syncwarp();
                if (c > 2 * NC) {
                    ptx::tma_load_2d_if(leader, st, &map_du, &sh->full[stage], 64 * (T::DU_ALL - 1), p0);
                } else if (c < 2 * NC) {
                    ptx::tma_load_3d_if(leader, st, &map_w, &sh->full[stage], 64 * (c >> 1), d0, c & 1);
                } else {
#pragma unroll
                    for (int q = 0; q < ND / 64; ++q)
                        ptx::tma_load_3d_if(leader, st + q * RP * 128, &map_a, &sh->full[stage], d0 + 64 * q, 0, g);
                }
                if (++stage == SLOTS) { stage = 0; phase ^= 1u; }
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = ptx::idesc_f16_f32(128, ND), idesc_u = ptx::idesc_bf16_f32(128, ND) | kIdescBMn;
        int stage = 0, buf = 0;
        uint32_t phase = 0, aphase = 0, bphase = 0;
        int64_t held = -1;
        int g = 0, p0 = 0, cnt = 0;
        bool ok = true;
        for (int64_t u = lo; ok && u < hi; ++u) {
            const int64_t tile = u / ndc;
            if (tile != held) {
                if (held >= 0 && cnt > 0) ptx::umma_commit_if(leader, &sh->aempty);  // the tile before has been read
                held = tile;
                cnt = rows_of(tile, g, p0);
                if (cnt > 0) {
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->afull, aphase, abort_flag));
                    if (!ok) break;
                    aphase ^= 1u;
                }
            }
            if (cnt == 0) continue;
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->tempty[buf], bphase ^ 1u, abort_flag));
            if (!ok) break;
            const uint32_t acc = tmem + (uint32_t)(buf * ND);
            for (int c = 0; c < 2 * NC + (g < na ? 1 : 0); ++c) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->full[stage], phase, abort_flag));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t st = ptx::smem_u32(ring + stage * T::SLOT);
                if (c < 2 * NC) {  // columns behind n are zero on both sides
                    const uint64_t ahi = ptx::sw128_kmajor_desc(ptx::smem_u32(sa + (c >> 1) * 16384));
                    const uint64_t alo = ptx::sw128_kmajor_desc(ptx::smem_u32(sa + (NC + (c >> 1)) * 16384));
                    const uint64_t bd = ptx::sw128_kmajor_desc(st);
#pragma unroll
                    for (int k = 0; k < 4; ++k) ptx::umma_bf16_if(leader, acc, ahi + 2 * k, bd + 2 * k, idesc, (c | k) != 0);
                    if ((c & 1) == 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) ptx::umma_bf16_if(leader, acc, alo + 2 * k, bd + 2 * k, idesc, 1u);
                    }
                } else {
                    const uint32_t ua = ptx::smem_u32(su);
                    const uint64_t u0 = ptx::sw128_kmajor_desc(ua);
                    const uint64_t u1 = RP == 32 ? u0 + 4 : ptx::sw128_kmajor_desc(ua + 16384);
                    const uint64_t bd = sw128_mnmajor_desc(st, RP * 128);
                    uint64_t u2 = ptx::sw128_kmajor_desc(ua + (T::DU_ALL - 1) * 16384);
                    const int held = stage;
                    if (T::STREAM) {
                        if (++stage == SLOTS) { stage = 0; phase ^= 1u; }
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->full[stage], phase, abort_flag));
                        if (!ok) break;
                        ptx::tc_fence_after();
                        u2 = ptx::sw128_kmajor_desc(ptx::smem_u32(ring + stage * T::SLOT));
                    }
#pragma unroll
                    for (int k = 0; k < RP / 16; ++k)
                        if (16 * k < r) {
                            ptx::umma_bf16_if(leader, acc, u0 + 2 * k, bd + 128 * k, idesc_u, 1u);
                            ptx::umma_bf16_if(leader, acc, u1 + 2 * k, bd + 128 * k, idesc_u, 1u);
                            ptx::umma_bf16_if(leader, acc, u2 + 2 * k, bd + 128 * k, idesc_u, 1u);
                        }
                    if (T::STREAM) ptx::umma_commit_if(leader, &sh->empty[held]);
                }
                ptx::umma_commit_if(leader, &sh->empty[stage]);
                if (++stage == SLOTS) { stage = 0; phase ^= 1u; }
            }
            ptx::umma_commit_if(leader, &sh->tfull[buf]);
            if (++buf == 2) { buf = 0; bphase ^= 1u; }
        }
    } else if (warp >= 4) {
        const int quad = warp & 3, grp = (warp - 4) >> 2;
        const int col0 = grp * (ND / 2);                  // the two warps of a quadrant share its columns
        uint8_t* mine = outs + (warp - 4) * 32 * 64 * 2;  // [32][64] bf16, 16-byte pieces swizzled by row
        constexpr int PIECES = 8;
        int buf = 0;
        uint32_t bphase = 0;
        int64_t held = -1;
        int g = 0, p0 = 0, cnt = 0;
        int32_t rows[PIECES];  // the rows that this lane stores: quad rows lane / PIECES + (32 / PIECES) i
        uint32_t rs[PIECES];   // 2^-k of these rows, twice
        for (int64_t u = lo; u < hi; ++u) {
            const int64_t tile = u / ndc;
            const int d0 = (int)(u - tile * ndc) * ND;
            if (tile != held) {
                held = tile;
                cnt = rows_of(tile, g, p0);
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const int q = quad * 32 + lane / PIECES + 32 / PIECES * i;
                    rows[i] = q < cnt ? plan.perm[p0 + q] : -1;
                    const __nv_bfloat162 two = __float2bfloat162_rn(q < cnt ? rinv[p0 + q] : 1.f);
                    rs[i] = *reinterpret_cast<const uint32_t*>(&two);
                }
            }
            if (cnt == 0) continue;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sh->tfull[buf], bphase, abort_flag))) break;
            ptx::tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * ND + col0);
            const bool any = quad * 32 < cnt;
            uint4 cs[ND / 128];  // 2^-k of the eight columns that this lane stores
#pragma unroll
            for (int w = 0; w < ND / 128; ++w)
                cs[w] = *reinterpret_cast<const uint4*>(cinv + d0 + col0 + 64 * w + 8 * (lane % PIECES));
#pragma unroll
            for (int w = 0; w < ND / 2; w += 64) {
                if (any) {
                    uint32_t v[64];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        ptx::tmem_ld16_issue(acc + (uint32_t)(w + 16 * q), *reinterpret_cast<uint32_t(*)[16]>(v + 16 * q));
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) {
                        uint32_t o[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[8 * p + 2 * q]), __uint_as_float(v[8 * p + 2 * q + 1]));
                            o[q] = *reinterpret_cast<const uint32_t*>(&b);
                        }
                        const int at = p ^ (lane & 7);
                        *reinterpret_cast<uint4*>(mine + (lane * PIECES + at) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                if (w + 64 >= ND / 2) {  // the accumulator is read
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&sh->tempty[buf]);
                }
                __syncwarp();
                if (any) {
                    const int piece = lane % PIECES, col = d0 + col0 + w + 8 * piece;
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) {
                        const int q = lane / PIECES + 32 / PIECES * i;
                        const int at = piece ^ (q & 7);
                        uint4 t = *reinterpret_cast<const uint4*>(mine + (q * PIECES + at) * 16);
                        const uint4 c = cs[w / 64];
                        t = make_uint4(mul_bf16x2(mul_bf16x2(t.x, rs[i]), c.x), mul_bf16x2(mul_bf16x2(t.y, rs[i]), c.y),
                                       mul_bf16x2(mul_bf16x2(t.z, rs[i]), c.z), mul_bf16x2(mul_bf16x2(t.w, rs[i]), c.w));
                        if (rows[i] >= 0 && col < d) *reinterpret_cast<uint4*>(dx + (int64_t)rows[i] * d + col) = t;
                    }
                }
                __syncwarp();
            }
            if (++buf == 2) { buf = 0; bphase ^= 1u; }
        }
    }
    ptx::settle_after_abort(abort_flag);
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 2 * ND);
    }
}

// ---------------------------------------------------------------- contraction over rows
namespace rct {
constexpr int kThreads = 384, kDrain = 4, kRun = 8, BD = 256, BK = adp::kPad;
}

struct RctShared {
    uint64_t full[4], empty[4], tfull, tempty;
    uint32_t tmem_base;
    int abort_flag, last;
};

// C columns of the other operand, in three bf16 parts: [p0 | p1], [p2] in chunks of 64 for C = 32, one
// chunk each for C = 64.
template <int C>
struct RctTile {
    static constexpr int CHUNKS = C == 32 ? 2 : 3;
    static constexpr int X_BYTES = 4 * rct::BK * 128, STAGE = X_BYTES + CHUNKS * rct::BK * 128;
    static constexpr int STAGES = 3, ACOLS = 3 * C;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + sizeof(RctShared);
};

// out[g][c][dd] (strides gs, cs, ds) = sum over the grouped positions p of group g of P[p][c] x[perm[p]][dd].
// A unit is (group, 256 columns of d, C columns of P); its K blocks are the group's blocks of 64 positions.
// `one`: all positions are one group. The line of K blocks is cut evenly over the CTAs, and a unit that a cut
// divides is finished by the last of its CTAs to arrive, in CTA order, as in router_adapters_tc_kernel.
// Padding positions have zero parts; their x rows are copies of a row of the same block, so that no other
// group's row (which might hold a NaN) meets a zero.
template <int C>
__global__ void __launch_bounds__(rct::kThreads, 1)
rows_contract_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                        const __grid_constant__ CUtensorMap map_p, int d, int ncols, int na, int one, AdapterPlan plan,
                        float* __restrict__ part, int32_t* __restrict__ tickets, float* __restrict__ out, int64_t gs,
                        int64_t cs, int64_t ds) {
    using namespace rct;
    using T = RctTile<C>;
    constexpr int STAGES = T::STAGES, ACOLS = T::ACOLS;
    constexpr uint32_t TCOLS = 2 * ACOLS <= 256 ? 256 : 512;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    RctShared* sh = reinterpret_cast<RctShared*>(smem + STAGES * T::STAGE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) { ptx::mbar_init(&sh->full[s], 3); ptx::mbar_init(&sh->empty[s], 1); }
        ptx::mbar_init(&sh->tfull, 1);
        ptx::mbar_init(&sh->tempty, 256);
        sh->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&map_x);
        ptx::prefetch_tensormap(&map_g);
        ptx::prefetch_tensormap(&map_p);
    }
    if (warp == 1) ptx::tmem_alloc(&sh->tmem_base, TCOLS);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    pdl_trigger();
    pdl_wait();
    const uint32_t tmem = sh->tmem_base;
    volatile int* abort_flag = &sh->abort_flag;
    const int ndt = (d + BD - 1) / BD, nct = (ncols + C - 1) / C, U = ndt * nct;
    const int64_t total = (int64_t)(plan.goff[one ? na + 1 : na] / BK) * U;
    // CTAs: runs of a unit's length on average, but not of more than kRun K blocks, while SMs are left (runs of 16 blocks
    // whatever the units were took 46 us for 100 rows of 40 adapters, d 2328: a CTA then had 16 units of one block each)
    int64_t units = U;
    if (!one) {
        int used = 0;
        for (int g0 = 0; g0 < na; g0 += kThreads)
            used += __syncthreads_count(g0 + tid < na && plan.goff[min(g0 + tid, na - 1) + 1] > plan.goff[min(g0 + tid, na - 1)]);
        units *= used;
    }
    int64_t run = units > 0 ? total / units : 1;
    run = run < 1 ? 1 : (run > kRun ? kRun : run);
    int64_t ctas = total / run;
    ctas = ctas < 1 ? 1 : (ctas > gridDim.x ? gridDim.x : ctas);
    const int64_t c = blockIdx.x;
    const int64_t lo = c < ctas ? c * total / ctas : total, hi = c < ctas ? (c + 1) * total / ctas : total;

    struct Unit {
        int g, dt, ct, blk0, nkb;  // blk0: the group's first block of 64 positions
        int64_t u0;                // the unit's first place on the line
    };
    auto unit_at = [&](int64_t pos) -> Unit {
        Unit u;
        u.g = 0;
        u.blk0 = 0;
        if (one) {
            u.nkb = plan.goff[na + 1] / BK;
        } else {
            u.g = group_at(plan.goff, na, (int)(pos / U) * BK);  // the last group that starts there: not empty
            u.blk0 = plan.goff[u.g] / BK;
            u.nkb = plan.goff[u.g + 1] / BK - u.blk0;
        }
        const int64_t in = pos - (int64_t)u.blk0 * U;
        const int q = (int)(in / u.nkb);
        u.dt = q / nct;
        u.ct = q % nct;
        u.u0 = (int64_t)u.blk0 * U + (int64_t)q * u.nkb;
        return u;
    };

    const uint32_t leader = lane == 0 ? 1u : 0u;
    if (warp < 4) {
        ptx::regs_less<72>();
        if (warp != 1) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t pos = lo; ok && pos < hi;) {
                const Unit u = unit_at(pos);
                const int kb0 = (int)(pos - u.u0), kb1 = (int)min((int64_t)u.nkb, kb0 + (hi - pos));
                const int slab = warp & 1, quad = lane & 7, chunk = lane >> 3;  // warps 2, 3: slab 0, 1
                // the block's first and last row of each slab and, in the gather warps, four rows a lane; the next
                // block's are on their way while this one is issued
                auto look = [&](int kb, int4& e, int4& v) {
                    const int32_t* q = plan.perm + (int64_t)(u.blk0 + kb) * BK;
                    e = make_int4(q[0], q[31], q[32], q[63]);
                    if (warp >= 2) v = *reinterpret_cast<const int4*>(q + 32 * slab + 4 * quad);
                };
                int4 edge, four = make_int4(0, 0, 0, 0), edge1, four1 = four;
                look(kb0, edge, four);
                for (int kb = kb0; kb < kb1; ++kb, edge = edge1, four = four1) {
                    const int p0 = (u.blk0 + kb) * BK;
                    if (kb + 1 < kb1) look(kb + 1, edge1, four1);
                    const int first0 = edge.x, first1 = edge.z;
                    const bool run0 = edge.y >= 0 && edge.y - first0 == 31, run1 = edge.w >= 0 && edge.w - first1 == 31;
                    const bool gather = warp >= 2 && !(slab == 0 ? run0 : run1);
                    const int rid[4] = {four.x < 0 ? first0 : four.x, four.y < 0 ? first0 : four.y,
                                        four.z < 0 ? first0 : four.z, four.w < 0 ? first0 : four.w};
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag));
                    if (!ok) break;
                    uint8_t* st = smem + stage * T::STAGE;
                    uint64_t* bar = &sh->full[stage];
                    // each of the three warps announces its own bytes, also none: a warp that a stage did not wait
                    // for could fall a whole ring behind and then wait for a phase that has passed
                    if (lane == 0)
                        ptx::mbar_expect_tx(bar, warp == 0 ? T::CHUNKS * BK * 128 + ((run0 ? 4 : 0) + (run1 ? 4 : 0)) * 4096
                                                           : (gather ? 16384 : 0));
                    __syncwarp();
                    if (warp == 0) {
#pragma unroll
                        for (int q = 0; q < T::CHUNKS; ++q)  // dh: a plane per part; du: the parts beside one another
                            ptx::tma_load_3d_if(leader, st + T::X_BYTES + q * BK * 128, &map_p, bar, one ? C * u.ct : 64 * q, p0, one ? q : 0);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (run0) ptx::tma_load_2d_if(leader, st + q * BK * 128, &map_x, bar, u.dt * BD + 64 * q, first0);
                            if (run1) ptx::tma_load_2d_if(leader, st + q * BK * 128 + 4096, &map_x, bar, u.dt * BD + 64 * q, first1);
                        }
                    } else if (gather) {
                        tma_gather4(st + chunk * BK * 128 + slab * 4096 + quad * 512, &map_g, bar, u.dt * BD + 64 * chunk, rid[0],
                                    rid[1], rid[2], rid[3]);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                pos += kb1 - kb0;
            }
        } else {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, ACOLS) | kIdescAMn | kIdescBMn;
            int stage = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            for (int64_t pos = lo; ok && pos < hi;) {
                const Unit u = unit_at(pos);
                const int kb0 = (int)(pos - u.u0), kb1 = (int)min((int64_t)u.nkb, kb0 + (hi - pos));
                const int halves = d - u.dt * BD > 128 ? 2 : 1;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const int in = (kb - kb0) % kDrain;
                    if (in == 0) {
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->tempty, tphase ^ 1u, abort_flag));
                        if (!ok) break;
                    }
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->full[stage], phase, abort_flag));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t st = ptx::smem_u32(smem + stage * T::STAGE);
                    const uint64_t bdesc = sw128_mnmajor_desc(st + T::X_BYTES, BK * 128);
                    for (int h = 0; h < halves; ++h) {
                        const uint64_t adesc = sw128_mnmajor_desc(st + h * 2 * BK * 128, BK * 128);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            ptx::umma_bf16_if(leader, tmem + (uint32_t)(h * ACOLS), adesc + 128 * kk, bdesc + 128 * kk, idesc,
                                           (in != 0 || kk != 0) ? 1u : 0u);
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
        const int row = half * 128 + quad * 32 + lane;  // column of the d tile
        const int et = tid - 128;
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * ACOLS);
        uint32_t tphase = 0;
        bool ok = true;
        for (int64_t pos = lo; pos < hi;) {
            const Unit u = unit_at(pos);
            const int kb0 = (int)(pos - u.u0), kb1 = (int)min((int64_t)u.nkb, kb0 + (hi - pos));
            const int dd = u.dt * BD + row;
            const bool mine = u.dt * BD + half * 128 < d;
            float acc[C];
#pragma unroll
            for (int j = 0; j < C; ++j) acc[j] = 0.f;
            for (int kb = kb0; kb < kb1; kb += kDrain) {
                // after a give-up every warp still walks its loops: the barriers below count them all
                if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&sh->tfull, tphase, abort_flag));
                tphase ^= 1u;
                if (!ok) continue;
                ptx::tc_fence_after();
                if (mine) {
#pragma unroll
                    for (int q = 0; q < C / 16; ++q) {
                        uint32_t v[3][16];
#pragma unroll
                        for (int p = 0; p < 3; ++p) ptx::tmem_ld16_issue(trow + (uint32_t)(p * C + q * 16), v[p]);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[q * 16 + j] = __fadd_rn(acc[q * 16 + j], __fadd_rn(__fadd_rn(__uint_as_float(v[2][j]), __uint_as_float(v[1][j])),
                                                                                   __uint_as_float(v[0][j])));
                    }
                }
                ptx::tc_fence_before();
                ptx::mbar_arrive(&sh->tempty);
            }
            bool finish = true;
            if (kb0 != 0 || kb1 != u.nkb) {
                float4* mp = reinterpret_cast<float4*>(part) + (2 * c + (kb0 == 0 ? 1 : 0)) * (int64_t)C / 4 * BD + row;
                if (ok && mine) {
#pragma unroll
                    for (int j = 0; j < C; j += 4) __stcg(mp + (int64_t)(j / 4) * BD, make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
                }
                __threadfence();
                ptx::named_barrier(1, 256);
                const int64_t cf = ((u.u0 + 1) * ctas + total - 1) / total - 1;
                const int64_t cl = ((u.u0 + u.nkb) * ctas + total - 1) / total - 1;
                if (et == 0) sh->last = atomicAdd(tickets + (int64_t)u.g * U + u.dt * nct + u.ct, 1) == (int)(cl - cf);
                ptx::named_barrier(1, 256);
                finish = sh->last != 0;
                if (finish) {
                    __threadfence();
#pragma unroll
                    for (int j = 0; j < C; ++j) acc[j] = 0.f;
                    if (mine) {
                        for (int64_t cc = cf; cc <= cl; ++cc) {
                            const int64_t at = cc * total / ctas;  // where the CTA's run begins
                            const float4* op = reinterpret_cast<const float4*>(part) + (2 * cc + (at <= u.u0 ? 1 : 0)) * (int64_t)C / 4 * BD + row;
#pragma unroll
                            for (int j = 0; j < C; j += 4) {
                                const float4 t = __ldcg(op + (int64_t)(j / 4) * BD);
                                acc[j] = __fadd_rn(acc[j], t.x); acc[j + 1] = __fadd_rn(acc[j + 1], t.y);
                                acc[j + 2] = __fadd_rn(acc[j + 2], t.z); acc[j + 3] = __fadd_rn(acc[j + 3], t.w);
                            }
                        }
                    }
                }
            }
            if (finish && ok && dd < d) {
                float* o = out + u.g * gs + (int64_t)u.ct * C * cs + dd * ds;
#pragma unroll
                for (int j = 0; j < C; ++j)
                    if (u.ct * C + j < ncols) o[j * cs] = acc[j];
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

// ---------------------------------------------------------------- host side
struct AgtWs {
    AdapterPlan plan;
    __half* wscaled;        // [2, d, nk]
    __nv_bfloat16* cinv;    // [d], padded to 256
    __nv_bfloat16* ascaled; // [na r, d]
    SplitOut split;
    float *slots;           // [grid + na][n, r]
    float *part;            // [2 kNumSMs][64][256]
    int32_t *tickets;       // one per unit of the two contractions
};

struct AgtShape {
    int nk, rp, pc, ndt, nct;
    int64_t mp, tickets_a, tickets_w;
};

static AgtShape agt_shape(int64_t m, int d, int n, int r, int na) {
    AgtShape s;
    s.nk = (n + 7) / 8 * 8;
    s.rp = r <= 32 ? 32 : 64;
    s.pc = r <= 32 ? 128 : 192;
    s.ndt = (d + rct::BD - 1) / rct::BD;
    s.nct = (n + 63) / 64;
    s.mp = adapter_padded_rows(m, na);
    s.tickets_a = (int64_t)na * s.ndt;
    s.tickets_w = (int64_t)s.ndt * s.nct;
    return s;
}

static size_t agt_layout(int64_t m, int d, int n, int r, int na, AgtWs* w, char* base) {
    const AgtShape s = agt_shape(m, d, n, r, na);
    size_t off = adapter_plan_layout(m, na, w ? &w->plan : nullptr, base);
    auto take = [&](size_t bytes) { char* p = base + off; off += (bytes + 255) & ~size_t(255); return p; };
    char* p;
    p = take((size_t)2 * d * s.nk * 2);                         if (w) w->wscaled = (__half*)p;
    p = take((size_t)(d + 255) / 256 * 256 * 2);                if (w) w->cinv = (__nv_bfloat16*)p;
    p = take((size_t)na * r * d * 2);                           if (w) w->ascaled = (__nv_bfloat16*)p;
    p = take((size_t)3 * s.mp * s.nk * 2);                      if (w) w->split.dhp = (__nv_bfloat16*)p;
    p = take((size_t)s.mp * s.pc * 2);                          if (w) w->split.dup = (__nv_bfloat16*)p;
    p = take((size_t)2 * s.mp * s.nk * 2);                      if (w) w->split.dhs = (__half*)p;
    p = take((size_t)s.mp * s.pc * 2);                          if (w) w->split.dus = (__nv_bfloat16*)p;
    p = take((size_t)s.mp * 4);                                 if (w) w->split.rinv = (float*)p;
    p = take((size_t)(asp::kGrid + na) * n * r * 4);            if (w) w->slots = (float*)p;
    p = take((size_t)2 * kNumSMs * 64 * rct::BD * 4);           if (w) w->part = (float*)p;
    p = take((size_t)(s.tickets_a + s.tickets_w) * 4);          if (w) w->tickets = (int32_t*)p;
    return off;
}

template <int ND, int NC, int RP>
static cudaError_t launch_adx(const CUtensorMap& mdh, const CUtensorMap& mdu, const CUtensorMap& mw,
                              const CUtensorMap& ma, int d, int r, int na, const AgtWs& w, __nv_bfloat16* dx,
                              cudaStream_t stream) {
    constexpr size_t smem = AdxTile<ND, NC, RP>::SMEM;
    const cudaError_t e = need_smem<adapters_dx_tc_kernel<ND, NC, RP>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(adapters_dx_tc_kernel<ND, NC, RP>, dim3(kNumSMs), dim3(adx::kThreads), smem, stream, mdh, mdu,
                      mw, ma, d, r, na, w.plan, w.split.rinv, w.cinv, dx);
}

template <int C>
static cudaError_t launch_rct(const CUtensorMap& mx, const CUtensorMap& mg, const CUtensorMap& mp, int d, int ncols,
                              int na, int one, const AdapterPlan& plan, float* part, int32_t* tickets, float* out,
                              int64_t gs, int64_t cs, int64_t ds, cudaStream_t stream) {
    constexpr size_t smem = RctTile<C>::SMEM;
    const cudaError_t e = need_smem<rows_contract_tc_kernel<C>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_contract_tc_kernel<C>, dim3(kNumSMs), dim3(rct::kThreads), smem, stream, mx, mg, mp, d, ncols,
                      na, one, plan, part, tickets, out, gs, cs, ds);
}

template <int NE, int NJ, int RP>
static cudaError_t launch_split(const float* dh, const float* hidden, const __nv_bfloat16* b, const float* scale, int n,
                                int r, int na, const AgtShape& s, const AgtWs& w, cudaStream_t stream) {
    constexpr size_t smem = sizeof(float) * ((size_t)(asp::kRows + RP) * (NE * 32 + 4) + (size_t)asp::kRows * (RP + 4));
    const cudaError_t e = need_smem<adapters_split_kernel<NE, NJ, RP>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(adapters_split_kernel<NE, NJ, RP>, dim3(asp::kGrid), dim3(asp::kThreads), smem, stream, dh, hidden,
                      b, scale, n, r, na, w.plan, s.nk, s.mp, w.split, w.slots);
}

static cudaError_t launch_adapters_grad_tc(const float* dh, const __nv_bfloat16* x, const float* w_r,
                                           const __nv_bfloat16* a, const __nv_bfloat16* b, const int32_t* idx,
                                           const float* scale, const float* hidden, int64_t m, int d, int n, int r,
                                           int na, __nv_bfloat16* dx, float* da, float* db, float* dw_r,
                                           void* workspace, cudaStream_t stream) {
    const AgtShape s = agt_shape(m, d, n, r, na);
    AgtWs w;
    agt_layout(m, d, n, r, na, &w, static_cast<char*>(workspace));
    PrepExtra extra = {};
    extra.w_r = w_r; extra.d = d; extra.n = n; extra.nk = s.nk; extra.wscaled = dx ? w.wscaled : nullptr;
    extra.cinv = w.cinv; extra.a = a; extra.ascaled = w.ascaled; extra.arows = na * r;
    cudaError_t e = launch_adapter_prep(idx, m, na, w.plan, w.tickets, s.tickets_a + s.tickets_w, extra, stream);
    if (e != cudaSuccess) return e;
    if (!dx) { w.split.dhs = nullptr; w.split.dus = nullptr; w.split.rinv = nullptr; }
    if (!dw_r) w.split.dhp = nullptr;
#define MOE_SPLIT(NE, NJ, RP) e = launch_split<NE, NJ, RP>(dh, hidden, b, scale, n, r, na, s, w, stream)
#define MOE_SPLIT_R(NE) do { if (r <= 16) MOE_SPLIT(NE, 2, 32); else if (r <= 32) MOE_SPLIT(NE, 4, 32); else MOE_SPLIT(NE, 8, 64); } while (0)
    if (n <= 64) MOE_SPLIT_R(2);
    else if (n <= 128) MOE_SPLIT_R(4);
    else MOE_SPLIT_R(8);
#undef MOE_SPLIT_R
#undef MOE_SPLIT
    if (e != cudaSuccess) return e;
    CUtensorMap mx, mg, ma, mw, mdh, mdu, mpw, mpa;
    if (!map_2d(&mx, x, (uint64_t)m, (uint64_t)d, 32) || !map_2d(&mg, x, (uint64_t)m, (uint64_t)d, 1) ||
        !map_3d(&mpa, w.split.dup, 1, (uint64_t)s.mp, (uint64_t)s.pc, rct::BK))
        return cudaErrorInvalidValue;
    if (dx) {
        const int nd = n <= 128 ? 256 : 128;
        if (!map_3d(&mw, w.wscaled, 2, (uint64_t)d, (uint64_t)s.nk, (uint32_t)nd) ||
            !map_3d(&ma, w.ascaled, (uint64_t)na, (uint64_t)r, (uint64_t)d, (uint32_t)s.rp) ||
            !map_3d(&mdh, w.split.dhs, 2, (uint64_t)s.mp, (uint64_t)s.nk, 128) ||
            !map_2d(&mdu, w.split.dus, (uint64_t)s.mp, (uint64_t)s.pc, 128))
            return cudaErrorInvalidValue;
#define MOE_ADX(ND, NC, RP) e = launch_adx<ND, NC, RP>(mdh, mdu, mw, ma, d, r, na, w, dx, stream)
        if (n <= 64) { if (s.rp == 32) MOE_ADX(256, 1, 32); else MOE_ADX(256, 1, 64); }
        else if (n <= 128) { if (s.rp == 32) MOE_ADX(256, 2, 32); else MOE_ADX(256, 2, 64); }
        else { if (s.rp == 32) MOE_ADX(128, 4, 32); else MOE_ADX(128, 4, 64); }
#undef MOE_ADX
        if (e != cudaSuccess) return e;
    }
    if (s.rp == 32)
        e = launch_rct<32>(mx, mg, mpa, d, r, na, 0, w.plan, w.part, w.tickets, da, (int64_t)r * d, d, 1, stream);
    else
        e = launch_rct<64>(mx, mg, mpa, d, r, na, 0, w.plan, w.part, w.tickets, da, (int64_t)r * d, d, 1, stream);
    if (e != cudaSuccess) return e;
    if (dw_r) {
        if (!map_3d(&mpw, w.split.dhp, 3, (uint64_t)s.mp, (uint64_t)s.nk, rct::BK)) return cudaErrorInvalidValue;
        e = launch_rct<64>(mx, mg, mpw, d, n, na, 1, w.plan, w.part, w.tickets + s.tickets_a, dw_r, 0, 1, n, stream);
        if (e != cudaSuccess) return e;
    }
    const int64_t per = (int64_t)n * r;
    return launch_pdl(adapters_fold_kernel, dim3((unsigned)((per + asp::kThreads - 1) / asp::kThreads), (unsigned)na),
                      dim3(asp::kThreads), 0, stream, w.slots, n, r, d, na, w.plan, scale, db, da);
}

}  // namespace moe
