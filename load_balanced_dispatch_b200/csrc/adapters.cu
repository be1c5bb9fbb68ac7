// adapters.cu -- the router projection with a low-rank adapter per request, forward and backward:
// the fp32 FMA kernels (fp32 activations, and the parts that both types share).
//
// "Switch Transformers paper review" (tildalice.io/?p=118), Switch Routing Step 1, h = x W_r, with
// the selective-precision recipe (logits in fp32). Row i of the batch belongs to a request whose
// adapter is a = adapter_idx[i] (-1: none):
//   u_i = A_a x_i  (r values, "hidden"),   h_i = x_i W_r + s_a B_a u_i.
// Backward, dh = dL/dh:
//   du_i = s_a B_a^T dh_i,  dx_i = W_r dh_i + A_a^T du_i,
//   dA_a = sum_{i in a} du_i x_i^T,  dB_a = s_a sum_{i in a} dh_i u_i^T,  dW_r = sum_i x_i dh_i^T.
#include <atomic>

#include "tc_ptx.cuh"

namespace moe {

namespace adp {
constexpr int kThreads = 256;
constexpr int kPad = 64;        // a group's rows are padded to this many in the grouped order
constexpr int kTile = 256;      // rows of a tensor-core row tile
constexpr int kPlanThreads = 1024;
constexpr int kCluster = 8;     // CTAs that group the rows of a large batch
constexpr int kPrepRows = 256;  // rows of the adapters that a block scales
constexpr int kClusterRows = 2048;  // above this many rows (one CTA: 6 us for 8191 rows, 62 us for 65536)
}  // namespace adp

// Rows grouped by adapter (group na: rows without one), in row order inside a group, each group
// padded to a multiple of kPad with -1.
struct AdapterPlan {
    int32_t *perm;   // [m_pad] row of each grouped position, or -1
    int32_t *goff;   // [na + 2] first grouped position of each group
    int32_t *gcnt;   // [na + 1] rows of each group
    int32_t *tstart; // [na + 2] first row tile (kTile grouped positions) of each group
};

static int64_t adapter_padded_rows(int64_t m, int na) { return m + (int64_t)adp::kPad * (na + 1); }

static size_t adapter_plan_layout(int64_t m, int na, AdapterPlan* plan, char* base) {
    size_t off = 0;
    auto take = [&](size_t ints) { char* p = base + off; off += (4 * ints + 255) & ~size_t(255); return (int32_t*)p; };
    int32_t* p;
    p = take((size_t)adapter_padded_rows(m, na)); if (plan) plan->perm = p;
    p = take((size_t)na + 2);                     if (plan) plan->goff = p;
    p = take((size_t)na + 1);                     if (plan) plan->gcnt = p;
    p = take((size_t)na + 2);                     if (plan) plan->tstart = p;
    return off;
}

// Largest g in [0, groups) with start[g] <= t.
__device__ __forceinline__ int group_at(const int32_t* __restrict__ start, int groups, int t) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// What the blocks behind the plan's do: parts of W_r for the tensor cores, or du for the fp32 kernels.
struct PrepExtra {
    const float* w_r;       // W_r [d, n] ...
    int d, n;
    __nv_bfloat16* wparts;  // ... for x W_r: three bf16 parts that add up to it, [3, n, d] (transposed)
    // ... for dh W_r^T: row t times 2^k_t as two fp16 parts [2, d, nk], nk >= n with zeros behind n; 2^-k_t; and the
    // adapters' columns t times 2^k_t, [na r, d], since their products are added to the same sums
    __half* wscaled;
    int nk, arows;
    __nv_bfloat16* cinv;
    const __nv_bfloat16* a;
    __nv_bfloat16* ascaled;
    const float *dh, *b, *scale;  // du_ij = s_a sum_e dh_ie B_a[e, j], a warp per row, lanes along j
    int r;
    float* du;
};

// k such that values of magnitude up to `top` are below 2^14 after a product with 2^k (top 0, inf or NaN: 0), at most
// `most`. Two fp16 parts then hold such a value to 2^-22 of itself or 2^-38 of the largest, and a product of two of
// them, or the sum of 256, is far from the ends of fp32.
__device__ __forceinline__ int fit_exponent(float top, int most) {
    if (!(top > 0.f) || isinf(top)) return 0;
    int e;
    frexpf(top, &e);  // top < 2^e
    return min(14 - e, most);
}
// The most for rows of dh and of W_r: 2^126 is the last with a normal reciprocal; an adapter's column is scaled with its
// row of W_r and may be far larger, so that stops where du A_a is still far from the end of fp32 (W_r's rows below 2^-60
// lose bits).
constexpr int kRowExponent = 126, kColExponent = 60;

// v to within 2^-22 of itself (or 2^-25)
__device__ __forceinline__ void split2h(float v, __half (&p)[2]) {
    p[0] = __float2half_rn(v);
    p[1] = __float2half_rn(v - __half2float(p[0]));
}

// Stable grouping of the rows by adapter by one cluster (blocks 0 .. its size - 1). Each warp takes a run of
// consecutive rows: a histogram per warp, sums over the warps and the CTAs before, then each warp places its rows;
// within 32 rows the lanes of one group rank themselves by a match. Block 0 also clears the tickets.
__global__ void __launch_bounds__(adp::kPlanThreads)
adapter_prep_kernel(const int32_t* __restrict__ idx, int64_t m, int na, AdapterPlan p, int32_t* __restrict__ tickets,
                    int64_t ntickets, PrepExtra x, int cluster) {
    using namespace adp;
    extern __shared__ int hist[];  // [32][G] per warp; [G] this CTA's counts; [G] all counts; [G] first position
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, G = na + 1;
    pdl_trigger();
    pdl_wait();
    if ((int)blockIdx.x >= cluster) {
        const int b = (int)blockIdx.x - cluster;
        if (x.du) {
            const int64_t row = (int64_t)b * 32 + wid;
            if (row >= m) return;
            const int ad = idx[row];
            const bool has = ad >= 0 && ad < na;
            for (int j = lane; j < x.r; j += 32) {
                float t = 0.f;
                if (has) {
                    const float* bp = x.b + (int64_t)ad * x.n * x.r + j;
#pragma unroll 8
                    for (int e = 0; e < x.n; ++e) t = fmaf(x.dh[row * x.n + e], bp[(int64_t)e * x.r], t);
                    t *= x.scale[ad];
                }
                x.du[row * x.r + j] = t;
            }
            return;
        }
        __shared__ float tile[32][33];
        const int d = x.d, n = x.n;
        if (x.wscaled) {  // rows t0 .. t0 + 31 of W_r, a warp each, and kPrepRows rows of the adapters in these columns
            const int nt = (d + 31) / 32, t0 = b % nt * 32, q0 = b / nt * kPrepRows, t = t0 + wid;
            if (q0 > 0 && q0 >= x.arows) return;
            float top = 0.f;
            if (t < d)
                for (int j = lane; j < n; j += 32) top = fmaxf(top, fabsf(x.w_r[(int64_t)t * n + j]));
            const int k = fit_exponent(warp_max(top), kColExponent);
            const float c = ldexpf(1.f, k);
            if (lane == 0) tile[0][wid] = c;
            if (q0 == 0 && t < d) {
                if (lane == 0) x.cinv[t] = __float2bfloat16_rn(ldexpf(1.f, -k));
                for (int j = lane; j < x.nk; j += 32) {
                    __half p[2];
                    split2h(j < n ? x.w_r[(int64_t)t * n + j] * c : 0.f, p);
                    x.wscaled[(int64_t)t * x.nk + j] = p[0];
                    x.wscaled[((int64_t)d + t) * x.nk + j] = p[1];
                }
            }
            __syncthreads();
            if (t0 + lane < d)
                for (int q = q0 + wid; q < min(q0 + kPrepRows, x.arows); q += 32)
                    x.ascaled[(int64_t)q * d + t0 + lane] =
                        __float2bfloat16_rn(__bfloat162float(x.a[(int64_t)q * d + t0 + lane]) * tile[0][lane]);
            return;
        }
        const int nb = (n + 31) / 32, t0 = b / nb * 32, j0 = b % nb * 32;
        if (t0 >= d) return;
        tile[wid][lane] = (t0 + wid < d && j0 + lane < n) ? x.w_r[(int64_t)(t0 + wid) * n + j0 + lane] : 0.f;
        __syncthreads();
        const int j = j0 + wid, t = t0 + lane;
        const float v = tile[lane][wid];
        if (j >= n || t >= d) return;
        const __nv_bfloat16 p0 = __float2bfloat16_rn(v);
        const float r1 = v - __bfloat162float(p0);
        const __nv_bfloat16 p1 = __float2bfloat16_rn(r1);
        const int64_t o = (int64_t)j * d + t, plane = (int64_t)n * d;
        x.wparts[o] = p0;
        x.wparts[plane + o] = p1;
        x.wparts[2 * plane + o] = __float2bfloat16_rn(r1 - __bfloat162float(p1));
        return;
    }
    int* own = hist + 32 * G;
    int* all = own + G;
    int* first = all + G;
    const int rank = blockIdx.x;
    for (int64_t i = (int64_t)rank * kPlanThreads + tid; i < ntickets; i += (int64_t)cluster * kPlanThreads) tickets[i] = 0;
    for (int i = tid; i < 32 * G; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const int64_t warps = 32 * cluster, per = ((m + warps - 1) / warps + 31) / 32 * 32;  // rows per warp, a multiple of 32
    const int64_t r0 = min((rank * 32 + wid) * per, m), r1 = min(r0 + per, m);
    int* mine = hist + wid * G;
    for (int64_t b = r0; b < r1; b += 128) {
        int g[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) g[q] = b + 32 * q + lane < r1 ? idx[b + 32 * q + lane] : -2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool in = b + 32 * q + lane < r1;
            if (in && (g[q] < -1 || g[q] >= na)) record_error(kErrAdapterIndex);
            const int v = !in ? -1 : (g[q] < 0 || g[q] >= na ? na : g[q]);
            const unsigned same = __match_any_sync(0xffffffffu, v);
            if (v >= 0 && lane == __ffs(same) - 1) mine[v] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int g = tid; g < G; g += kPlanThreads) {
        int c = 0;
        for (int w = 0; w < 32; ++w) c += hist[w * G + g];
        own[g] = c;
    }
    if (cluster > 1) ptx::cluster_sync(); else __syncthreads();
    for (int g = tid; g < G; g += kPlanThreads) {
        int sum = 0, before = 0;
        for (int k = 0; k < cluster; ++k) {
            const int c = cluster > 1 ? ptx::ld_cluster_s32(ptx::mapa_shared(ptx::smem_u32(own + g), k)) : own[g];
            sum += c;
            if (k < rank) before += c;
        }
        all[g] = sum;
        first[g] = before;
    }
    __syncthreads();
    if (wid == 0) {
        int base = 0, til = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            const int c = g < G ? all[g] : 0;
            const int pc = (c + kPad - 1) / kPad * kPad, tc = (pc + kTile - 1) / kTile;
            int a = pc, t = tc;
            for (int o = 1; o < 32; o <<= 1) {
                const int ua = __shfl_up_sync(0xffffffffu, a, o), ut = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) { a += ua; t += ut; }
            }
            if (g < G) {
                first[g] += base + a - pc;
                if (rank == 0) { p.goff[g] = base + a - pc; p.gcnt[g] = c; p.tstart[g] = til + t - tc; }
            }
            base += __shfl_sync(0xffffffffu, a, 31);
            til += __shfl_sync(0xffffffffu, t, 31);
        }
        if (rank == 0 && lane == 0) { p.goff[G] = base; p.tstart[G] = til; }
    }
    __syncthreads();
    for (int g = tid; g < G; g += kPlanThreads) {
        int at = first[g];
        for (int w = 0; w < 32; ++w) { const int c = hist[w * G + g]; hist[w * G + g] = at; at += c; }
        if (rank == cluster - 1)  // behind the group's last row
            for (int q = all[g]; q % kPad != 0; ++q) p.perm[at++] = -1;
    }
    __syncthreads();
    for (int64_t b = r0; b < r1; b += 128) {
        int g[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) g[q] = b + 32 * q + lane < r1 ? idx[b + 32 * q + lane] : -2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t r = b + 32 * q + lane;
            const int v = r >= r1 ? -1 : (g[q] < 0 || g[q] >= na ? na : g[q]);
            const unsigned same = __match_any_sync(0xffffffffu, v);
            const int place = __popc(same & ((1u << lane) - 1u));
            const int at = v >= 0 ? mine[v] : 0;
            __syncwarp();
            if (v >= 0) {
                p.perm[at + place] = (int32_t)r;
                if (place == 0) mine[v] = at + __popc(same);
            }
            __syncwarp();
        }
    }
    if (cluster > 1) ptx::cluster_sync();  // nobody leaves while its counts may still be read
}

// Set a kernel's shared-memory limit, once per device (the attribute belongs to the device).
template <auto Kernel>
static cudaError_t need_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1u))) return e;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    return e;
}

static cudaError_t launch_adapter_prep(const int32_t* idx, int64_t m, int na, const AdapterPlan& p, int32_t* tickets,
                                       int64_t ntickets, const PrepExtra& x, cudaStream_t stream) {
    const size_t per = sizeof(int) * 35;  // bytes per group
    const cudaError_t e = need_smem<adapter_prep_kernel>(per * (kMaxAdapters + 1));
    if (e != cudaSuccess) return e;
    const int cluster = m > adp::kClusterRows ? adp::kCluster : 1;
    int64_t extra = 0;
    if (x.wparts) extra = (int64_t)((x.d + 31) / 32) * ((x.n + 31) / 32);
    if (x.wscaled) extra = (int64_t)((x.d + 31) / 32) * ((x.arows + adp::kPrepRows - 1) / adp::kPrepRows);
    if (x.du) extra = (m + 31) / 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cluster + (extra + cluster - 1) / cluster * cluster));
    cfg.blockDim = dim3(adp::kPlanThreads);
    cfg.dynamicSmemBytes = per * (size_t)(na + 1);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adapter_prep_kernel, idx, m, na, p, tickets, ntickets, x, cluster);
}

// ---- forward of four rows by a cluster of 1 to 8 CTAs that shares out the columns of d: all fp32 batches, and bf16
// batches of few rows (adapters_run.cu has the rule). In a CTA, eight warps read its slice of W_r once for the four
// rows (a thread: four columns, every KL-th row of the slice) and eight form u (a warp: four products at a time, lanes
// along d; A_a is read once for the rows when they share it). These are other warps (512 threads) while all clusters
// surely run at once and W_r is not the larger part, and the same ones (256 threads, three CTAs per SM) for more rows:
// 8 against 11 us for 32 rows of 2048 columns, but 102 against 54 us for 4096 rows of 512. The slices' sums meet in
// distributed shared memory, where each CTA finishes a part of the columns. Nothing is grouped and one launch does
// all, so a step of few rows is bound by the latency of that chain, a large batch by the reads of A_a and W_r from L2.
constexpr int kFewRows = 4, kFewSlice = 512;  // rows of a cluster; columns of d in shared memory at a time

// Sums of four values over the warp, in six shuffles: lane l gets the sum of t[l / 8].
__device__ __forceinline__ float warp_sum4(const float (&t)[4], int lane) {
    float a = lane & 16 ? t[2] : t[0], b = lane & 16 ? t[3] : t[1];
    a += __shfl_xor_sync(0xffffffffu, lane & 16 ? t[0] : t[2], 16);
    b += __shfl_xor_sync(0xffffffffu, lane & 16 ? t[1] : t[3], 16);
    float c = (lane & 8 ? b : a) + __shfl_xor_sync(0xffffffffu, lane & 8 ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
}

template <typename T, int TH>
__global__ void __launch_bounds__(TH, TH == 256 ? 3 : 1)
adapters_few_kernel(const T* __restrict__ x, const float* __restrict__ w_r, const T* __restrict__ a,
                    const T* __restrict__ bmat, const int32_t* __restrict__ idx, const float* __restrict__ scale,
                    int64_t m, int d, int n, int r, int na, int cluster, float* __restrict__ logits,
                    float* __restrict__ hidden) {
    constexpr int V = Vec16<T>::N, kThreads = TH, WT = 256, W = 8;
    __shared__ float xs[kFewRows][kFewSlice];
    __shared__ float4 red[kFewRows][WT];                          // a thread's four columns of each row
    __shared__ float sl[kFewRows][kMaxExperts], su[kFewRows][kMaxRank];  // this slice's sums (read by the cluster)
    __shared__ float us[kFewRows][kMaxRank];                      // s u, complete
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int uw = TH == 512 ? wid - W : wid;  // which of the warps that form u
    pdl_trigger();
    pdl_wait();
    const int rank = (int)blockIdx.x % cluster;
    const int64_t row0 = (int64_t)(blockIdx.x / cluster) * kFewRows;
    const int rows = (int)min((int64_t)kFewRows, m - row0);
    const int per = (d / V + cluster - 1) / cluster * V;          // columns of a slice, whole 16-byte pieces
    const int k0 = min(rank * per, d), k1 = min(k0 + per, d);
    int ad[kFewRows];
#pragma unroll
    for (int q = 0; q < kFewRows; ++q) ad[q] = q < rows ? idx[row0 + q] : -1;
#pragma unroll
    for (int q = 0; q < kFewRows; ++q)
        if (ad[q] < -1 || ad[q] >= na) {
            if (tid == 0 && rank == 0) record_error(kErrAdapterIndex);
            ad[q] = -1;
        }
    const bool shared = ad[0] >= 0 && ad[0] == ad[1] && ad[0] == ad[2] && ad[0] == ad[3];
    const int cq = (n + 3) / 4, kl = WT / cq, col = tid % cq, kg = tid / cq;
    const bool vec = (n & 3) == 0, mine = tid < WT && kg < kl;
    float4 acc[kFewRows];
#pragma unroll
    for (int q = 0; q < kFewRows; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = tid; i < kFewRows * r; i += kThreads) su[i / r][i % r] = 0.f;
    for (int c0 = k0; c0 < k1; c0 += kFewSlice) {
        const int len = min(kFewSlice, k1 - c0);
        __syncthreads();
        for (int i = tid; i < kFewRows * (kFewSlice / V); i += kThreads) {
            const int q = i / (kFewSlice / V), c = i % (kFewSlice / V) * V;
            if (c >= len) continue;
            float v[V];
#pragma unroll
            for (int u = 0; u < V; ++u) v[u] = 0.f;
            if (q < rows) Vec16<T>::load(x + (row0 + q) * d + c0 + c, v);
#pragma unroll
            for (int u = 0; u < V; ++u) xs[q][c + u] = v[u];
        }
        __syncthreads();
        if (mine) {
            const float* wp = w_r + (int64_t)c0 * n + 4 * col;
#pragma unroll 8
            for (int k = kg; k < len; k += kl) {
                float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                const float* src = wp + (int64_t)k * n;
                if (vec) {
                    w = *reinterpret_cast<const float4*>(src);
                } else {
                    w.x = src[0];
                    if (4 * col + 1 < n) w.y = src[1];
                    if (4 * col + 2 < n) w.z = src[2];
                    if (4 * col + 3 < n) w.w = src[3];
                }
#pragma unroll
                for (int q = 0; q < kFewRows; ++q) {
                    const float xv = xs[q][k];
                    acc[q].x = fmaf(xv, w.x, acc[q].x);
                    acc[q].y = fmaf(xv, w.y, acc[q].y);
                    acc[q].z = fmaf(xv, w.z, acc[q].z);
                    acc[q].w = fmaf(xv, w.w, acc[q].w);
                }
            }
        }
        if (uw >= 0 && shared) {  // a rank at a time, its product with each row
#pragma unroll 4
            for (int j = uw; j < r; j += W) {
                const T* ap = a + ((int64_t)ad[0] * r + j) * d + c0;
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                for (int c = lane * V; c < len; c += 32 * V) {
                    float v[V];
                    Vec16<T>::load(ap + c, v);
#pragma unroll
                    for (int p = 0; p < 4; ++p)
#pragma unroll
                        for (int u = 0; u < V; ++u) t[p] = fmaf(xs[p][c + u], v[u], t[p]);
                }
                const float sum = warp_sum4(t, lane);
                if ((lane & 7) == 0) su[lane >> 3][j] += sum;
            }
        } else if (uw >= 0) {  // products i = (row, rank), a warp takes i0, i0 + W, ...: four at a time
            for (int i0 = uw; i0 < kFewRows * r; i0 += 4 * W) {
                float t[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int i = i0 + p * W, q = i / r, j = i - q * r;
                    t[p] = 0.f;
                    const int own = q == 0 ? ad[0] : q == 1 ? ad[1] : q == 2 ? ad[2] : ad[3];
                    if (i < kFewRows * r && own >= 0) {
                        const T* ap = a + ((int64_t)own * r + j) * d + c0;
                        for (int c = lane * V; c < len; c += 32 * V) {
                            float v[V];
                            Vec16<T>::load(ap + c, v);
#pragma unroll
                            for (int u = 0; u < V; ++u) t[p] = fmaf(xs[q][c + u], v[u], t[p]);
                        }
                    }
                }
                const float sum = warp_sum4(t, lane);
                const int i = i0 + (lane >> 3) * W;
                if ((lane & 7) == 0 && i < kFewRows * r) su[i / r][i % r] += sum;
            }
        }
    }
    if (mine) {
#pragma unroll
        for (int q = 0; q < kFewRows; ++q) red[q][kg * cq + col] = acc[q];
    }
    __syncthreads();
    for (int i = tid; i < kFewRows * cq; i += kThreads) {
        const int q = i / cq, c = i % cq;
        float4 t = red[q][c];
#pragma unroll 8
        for (int k = 1; k < kl; ++k) {
            const float4 v = red[q][k * cq + c];
            t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
        }
        *reinterpret_cast<float4*>(&sl[q][4 * c]) = t;
    }
    if (cluster > 1) ptx::cluster_sync(); else __syncthreads();
    for (int i = tid; i < rows * r; i += kThreads) {
        const int q = i / r, j = i % r;
        float t = 0.f;
        for (int k = 0; k < cluster; ++k)
            t += cluster > 1 ? ptx::ld_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&su[q][j]), k)) : su[q][j];
        if (rank == 0 && hidden) hidden[(row0 + q) * r + j] = t;
        us[q][j] = ad[q] >= 0 ? scale[ad[q]] * t : 0.f;
    }
    __syncthreads();
    for (int i = rank * kThreads + tid; i < rows * n; i += cluster * kThreads) {
        const int q = i / n, e = i % n;
        float t = 0.f;
        for (int k = 0; k < cluster; ++k)
            t += cluster > 1 ? ptx::ld_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&sl[q][e]), k)) : sl[q][e];
        if (ad[q] >= 0) {
            const T* bp = bmat + ((int64_t)ad[q] * n + e) * r;
            float v = 0.f;
            if (r % V == 0) {
#pragma unroll 2
                for (int j = 0; j < r; j += V) {
                    float bv[V];
                    Vec16<T>::load(bp + j, bv);
#pragma unroll
                    for (int u = 0; u < V; ++u) v = fmaf(us[q][j + u], bv[u], v);
                }
            } else {
#pragma unroll 8
                for (int j = 0; j < r; ++j) v = fmaf(us[q][j], Elem<T>::load(bp + j), v);
            }
            t += v;
        }
        logits[(row0 + q) * n + e] = t;
    }
    if (cluster > 1) ptx::cluster_sync();  // nobody leaves while its sums may still be read
}

template <typename T>
static cudaError_t launch_adapters_few(const T* x, const float* w_r, const T* a, const T* b, const int32_t* idx,
                                       const float* scale, int64_t m, int d, int n, int r, int na, float* logits,
                                       float* hidden, cudaStream_t stream) {
    int cluster = 1;
    while (cluster < 8 && d / cluster > 256) cluster *= 2;  // slices of 256 columns or so
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((m + kFewRows - 1) / kFewRows * cluster));
    const bool at_once = cfg.gridDim.x <= (unsigned)kNumSMs * 3 / 4 && n <= 128;
    cfg.blockDim = dim3(at_once ? 512 : 256);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, at_once ? adapters_few_kernel<T, 512> : adapters_few_kernel<T, 256>, x, w_r, a, b, idx, scale, m, d, n, r, na, cluster, logits,
                              hidden);
}

// ---- dx: 16 rows x 128 columns of d per CTA
__global__ void __launch_bounds__(adp::kThreads)
adapters_dx_kernel(const float* __restrict__ dh, const float* __restrict__ w_r, const float* __restrict__ a,
                   const int32_t* __restrict__ idx, const float* __restrict__ du, int64_t m, int d, int n, int r,
                   int na, float* __restrict__ dx) {
    using namespace adp;
    constexpr int R = 16, DC = 128, EC = 32;
    __shared__ float hs[R][kMaxExperts + 1];
    __shared__ float us[R][kMaxRank + 1];
    __shared__ float ws[EC][DC + 1];
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int64_t row0 = (int64_t)blockIdx.x * R;
    const int c0 = blockIdx.y * DC, col = tid % DC, rg = tid / DC;  // two row groups of eight
    for (int i = tid; i < R * n; i += kThreads) {
        const int64_t row = row0 + i / n;
        hs[i / n][i % n] = row < m ? dh[row * n + i % n] : 0.f;
    }
    for (int i = tid; i < R * r; i += kThreads) {
        const int64_t row = row0 + i / r;
        us[i / r][i % r] = row < m ? du[row * r + i % r] : 0.f;
    }
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
    for (int e0 = 0; e0 < n; e0 += EC) {
        __syncthreads();
        for (int i = tid; i < EC * DC; i += kThreads) {
            const int kk = i / EC, e = i % EC;
            ws[e][kk] = (c0 + kk < d && e0 + e < n) ? w_r[(int64_t)(c0 + kk) * n + e0 + e] : 0.f;
        }
        __syncthreads();
        const int top = min(EC, n - e0);
        for (int e = 0; e < top; ++e) {
            const float wv = ws[e][col];
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = fmaf(hs[rg * 8 + q][e0 + e], wv, acc[q]);
        }
    }
    if (c0 + col >= d) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int64_t row = row0 + rg * 8 + q;
        if (row >= m) continue;
        const int ad = idx[row];
        float t = 0.f;
        if (ad >= 0 && ad < na) {
            const float* ap = a + (int64_t)ad * r * d + c0 + col;
            for (int j = 0; j < r; ++j) t = fmaf(us[rg * 8 + q][j], ap[(int64_t)j * d], t);
        }
        dx[row * d + c0 + col] = acc[q] + t;
    }
}

// ---- row contractions out[g][q][p] = s_g sum over the rows of group g of X[row][p] Y[row][q].
// A segment is what a window of `seg` grouped positions has of one group: window w and group g give segment w + g
// (unique: each next segment advances the window or the group). Its partial sums are left as part[segment][q][p] and
// folded in order.
struct RowsTask {
    const float *X, *Y, *scale;
    int np, nq, seg, grouped;  // grouped 0: the rows in order, one group
    int ptiles, qtiles;
    int64_t segs;
    float *part, *out;
};
struct RowsTasks {
    RowsTask t[3];
    int count;
};

// 64 x 64 tiles, 4 x 4 per thread, 64 rows at a time; 16 rows' products are summed first and then added.
__global__ void __launch_bounds__(adp::kThreads)
rows_outer_kernel(RowsTasks tasks, int64_t m, int groups, AdapterPlan plan) {
    using namespace adp;
    constexpr int RB = 64;
    __shared__ float xs[RB][65], ys[RB][65];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, c = tid & 63;
    pdl_trigger();
    pdl_wait();
    int64_t blk = blockIdx.x;
    int ti = 0;
    while (ti + 1 < tasks.count && blk >= (int64_t)tasks.t[ti].ptiles * tasks.t[ti].qtiles * tasks.t[ti].segs) {
        blk -= (int64_t)tasks.t[ti].ptiles * tasks.t[ti].qtiles * tasks.t[ti].segs;
        ++ti;
    }
    const RowsTask& T = tasks.t[ti];
    const int p0 = (int)(blk % T.ptiles) * 64, q0 = (int)(blk / T.ptiles % T.qtiles) * 64;
    const int64_t seg = blk / ((int64_t)T.ptiles * T.qtiles);
    int64_t b = seg * T.seg, end = min(b + T.seg, m);
    if (T.grouped) {
        int lo = 0, hi = groups;  // largest group whose first segment is <= seg
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (plan.goff[mid] / T.seg + mid <= seg) lo = mid; else hi = mid;
        }
        if (lo == groups - 1) return;  // rows without an adapter: nobody reads their sums
        const int64_t w = seg - lo;
        b = max(w * T.seg, (int64_t)plan.goff[lo]);
        end = min((w + 1) * T.seg, (int64_t)plan.goff[lo + 1]);
    }
    if (b >= end) return;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int64_t at = b; at < end; at += RB) {
        int32_t row[RB / 4];
#pragma unroll
        for (int i = 0; i < RB / 4; ++i) {
            const int64_t q = at + (tid >> 6) + 4 * i;
            row[i] = q < end ? (T.grouped ? plan.perm[q] : (int32_t)q) : -1;
        }
#pragma unroll
        for (int i = 0; i < RB / 4; ++i) {
            xs[(tid >> 6) + 4 * i][c] = (row[i] >= 0 && p0 + c < T.np) ? T.X[(int64_t)row[i] * T.np + p0 + c] : 0.f;
            ys[(tid >> 6) + 4 * i][c] = (row[i] >= 0 && q0 + c < T.nq) ? T.Y[(int64_t)row[i] * T.nq + q0 + c] : 0.f;
        }
        __syncthreads();
        for (int r0 = 0; r0 < RB; r0 += 16) {
            float blk4[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) blk4[i][j] = 0.f;
#pragma unroll
            for (int rr = 0; rr < 16; ++rr) {
                float xv[4], yv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) { xv[i] = xs[r0 + rr][tx + 16 * i]; yv[i] = ys[r0 + rr][ty + 16 * i]; }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) blk4[i][j] = fmaf(xv[j], yv[i], blk4[i][j]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += blk4[i][j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = p0 + tx + 16 * j, q = q0 + ty + 16 * i;
            if (p < T.np && q < T.nq) T.part[(seg * T.nq + q) * T.np + p] = acc[i][j];
        }
}

// out[g][i] = s_g * sum over the group's segments, in order, of part[segment][i] (zero for no rows).
// blockIdx.y = group; blockIdx.x runs over the tasks' outputs.
__global__ void __launch_bounds__(adp::kThreads)
rows_fold_kernel(RowsTasks tasks, AdapterPlan plan) {
    pdl_trigger();
    pdl_wait();
    const int g = blockIdx.y;
    int64_t blk = blockIdx.x;
    int ti = 0;
    while (ti + 1 < tasks.count) {
        const int64_t mine = ((int64_t)tasks.t[ti].np * tasks.t[ti].nq + adp::kThreads - 1) / adp::kThreads;
        if (blk < mine) break;
        blk -= mine;
        ++ti;
    }
    const RowsTask& T = tasks.t[ti];
    const int64_t per = (int64_t)T.np * T.nq, i = blk * adp::kThreads + threadIdx.x;
    if (i >= per || (!T.grouped && g > 0)) return;
    int64_t s0 = 0, s1 = T.segs;
    if (T.grouped) {
        const int o0 = plan.goff[g], o1 = plan.goff[g + 1];
        s0 = o0 / T.seg + g;
        s1 = o1 > o0 ? (o1 - 1) / T.seg + g + 1 : s0;
    }
    float t = 0.f;
#pragma unroll 4
    for (int64_t s = s0; s < s1; ++s) t += T.part[s * per + i];
    T.out[g * per + i] = T.scale ? T.scale[g] * t : t;
}

// A task over `rows` (grouped: padded) rows. Segments of 64 rows, longer where their partial sums would take more
// than 16 MB.
static RowsTask rows_task(const float* X, int np, const float* Y, int nq, int64_t rows, int groups, bool grouped) {
    RowsTask t = {};
    t.X = X; t.Y = Y; t.np = np; t.nq = nq; t.grouped = grouped ? 1 : 0;
    t.ptiles = (np + 63) / 64;
    t.qtiles = (nq + 63) / 64;
    t.seg = 64;
    while ((int64_t)t.seg < rows && (rows / t.seg) * np * nq * 4 > ((int64_t)16 << 20)) t.seg *= 2;
    t.segs = (rows + t.seg - 1) / t.seg + (grouped ? groups : 0);
    return t;
}

struct AdapterWs {
    AdapterPlan plan;
    float* du;       // [m, r]
    RowsTask task[3];  // dA, dB, dW_r
};

static size_t adapter_ws_layout(int64_t m, int d, int n, int r, int na, AdapterWs* w, char* base) {
    size_t off = adapter_plan_layout(m, na, w ? &w->plan : nullptr, base);
    auto take = [&](size_t bytes) { char* p = base + off; off += (bytes + 255) & ~size_t(255); return p; };
    char* p;
    p = take(4 * (size_t)m * r);       if (w) w->du = (float*)p;
    const int64_t mp = adapter_padded_rows(m, na);
    RowsTask t[3] = {rows_task(nullptr, d, nullptr, r, mp, na + 1, true), rows_task(nullptr, r, nullptr, n, mp, na + 1, true),
                     rows_task(nullptr, n, nullptr, d, m, 1, false)};
    for (int i = 0; i < 3; ++i) {
        p = take(4 * (size_t)t[i].segs * t[i].np * t[i].nq);
        t[i].part = (float*)p;
        if (w) w->task[i] = t[i];
    }
    return off;
}

}  // namespace moe
