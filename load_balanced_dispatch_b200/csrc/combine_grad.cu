// combine_grad.cu -- backward of the combine y_i = (residual_i) + sum_r g_ir ybuf[dest_row[i, r]]
// ("Switch Transformer read for implementation", molayo1419.me: restore token order and multiply by
// the gate; "Switch Transformers paper review", Step 3, y = p_i* E_i*(x): the router learns through
// the gate):
//   dgate_ir = <dy_i, ybuf[dest_row[i, r]]>,   dybuf[dest_row[i, r]] = g_ir dy_i   (0 / no row for a drop).
// The gate is the one the combine multiplies by (rounded to bf16 in a bf16 layer). The residual's
// gradient is dy itself.
//
// One pass: dy and the kept rows of ybuf are read once, dybuf is written once, so HBM bounds it
// (5 m d elements for two kept picks). A warp holds a token: per 16-byte column chunk it loads dy
// and its picks' rows together, then adds the products in fp32 (a fixed order: lane partials over
// the chunks, then the warp's butterfly) and stores the scaled dy.
#include "common.cuh"

namespace moe {

namespace cgrad {
constexpr int kThreads = 256;
}

// U column chunks in flight per lane, picks in batches of KB (one batch when k <= KB).
template <typename T, int KB, int U>
__global__ void __launch_bounds__(cgrad::kThreads)
combine_grad_kernel(const T* __restrict__ dy, const T* __restrict__ ybuf, const int32_t* __restrict__ dest_row,
                    const float* __restrict__ gate, int64_t m, int k, int d, int64_t max_rows, int gate_bf16,
                    T* __restrict__ dybuf, float* __restrict__ dgate) {
    constexpr int V = Vec16<T>::N;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const int nvec = d / V;
    const int64_t warps = (int64_t)gridDim.x * (cgrad::kThreads / 32);
    for (int64_t i = (int64_t)blockIdx.x * (cgrad::kThreads / 32) + (threadIdx.x >> 5); i < m; i += warps) {
        const T* dyr = dy + i * d;
        for (int b = 0; b < k; b += KB) {
            int32_t myrow = -1;
            float myg = 0.f;
            if (lane < KB && b + lane < k) {
                myrow = dest_row[i * k + b + lane];
                myg = gate[i * k + b + lane];
                if (gate_bf16) myg = round_to_bf16(myg);
                if (myrow >= max_rows) { record_error(kErrRowOverflow); myrow = -1; }
            }
            int32_t rows[KB];
            float gs[KB], dot[KB];
#pragma unroll
            for (int r = 0; r < KB; ++r) {
                rows[r] = __shfl_sync(0xffffffffu, myrow, r);
                gs[r] = __shfl_sync(0xffffffffu, myg, r);
                dot[r] = 0.f;
            }
            for (int c0 = lane; c0 < nvec; c0 += 32 * U) {
                uint4 raw[U], row[KB][U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + 32 * u;
                    if (c < nvec) raw[u] = *reinterpret_cast<const uint4*>(dyr + (int64_t)c * V);
                }
#pragma unroll
                for (int r = 0; r < KB; ++r)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int c = c0 + 32 * u;
                        if (rows[r] >= 0 && c < nvec)
                            row[r][u] = *reinterpret_cast<const uint4*>(ybuf + (int64_t)rows[r] * d + (int64_t)c * V);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = c0 + 32 * u;
                    if (c >= nvec) continue;
                    float v[V], o[V], y[V];
                    Vec16<T>::load(reinterpret_cast<const T*>(&raw[u]), v);
#pragma unroll
                    for (int r = 0; r < KB; ++r) {
                        if (rows[r] < 0) continue;
                        Vec16<T>::load(reinterpret_cast<const T*>(&row[r][u]), y);
#pragma unroll
                        for (int q = 0; q < V; ++q) {
                            dot[r] = fmaf(v[q], y[q], dot[r]);
                            o[q] = gs[r] * v[q];
                        }
                        if (dybuf) Vec16<T>::store(dybuf + (int64_t)rows[r] * d + (int64_t)c * V, o);
                    }
                }
            }
            float out = 0.f;
#pragma unroll
            for (int r = 0; r < KB; ++r) {
                const float t = warp_sum(dot[r]);
                if (lane == r) out = t;
            }
            if (lane < KB && b + lane < k) dgate[i * k + b + lane] = out;
        }
    }
    pdl_trigger();
}

template <typename T>
static cudaError_t launch_combine_grad_t(const void* dy, const void* ybuf, const int32_t* dest_row, const float* gate,
                                         int64_t m, int k, int d, int64_t max_rows, int gate_bf16, void* dybuf,
                                         float* dgate, cudaStream_t stream) {
    const int64_t warps = cgrad::kThreads / 32;
    int64_t blocks = (m + warps - 1) / warps;
    if (blocks > (int64_t)kNumSMs * 64) blocks = (int64_t)kNumSMs * 64;
#define MOE_COMBINE_GRAD(KB, U)                                                                                       \
    launch_pdl(combine_grad_kernel<T, KB, U>, dim3((unsigned)blocks), dim3(cgrad::kThreads), 0, stream,               \
               static_cast<const T*>(dy), static_cast<const T*>(ybuf), dest_row, gate, m, k, d, max_rows, gate_bf16, \
               static_cast<T*>(dybuf), dgate)
    if (k == 1) return MOE_COMBINE_GRAD(1, 2);
    if (k == 2) return MOE_COMBINE_GRAD(2, 2);
    return MOE_COMBINE_GRAD(4, 2);
#undef MOE_COMBINE_GRAD
}

cudaError_t launch_combine_grad(const void* dy, const void* ybuf, moe_dtype dt, const int32_t* dest_row,
                                const float* gate, int64_t m, int k, int d, int64_t max_rows, void* dybuf,
                                float* dgate, cudaStream_t stream) {
    if (m == 0) return cudaSuccess;
    if (dt == MOE_BF16)
        return launch_combine_grad_t<__nv_bfloat16>(dy, ybuf, dest_row, gate, m, k, d, max_rows, 1, dybuf, dgate, stream);
    return launch_combine_grad_t<float>(dy, ybuf, dest_row, gate, m, k, d, max_rows, 0, dybuf, dgate, stream);
}

}  // namespace moe
