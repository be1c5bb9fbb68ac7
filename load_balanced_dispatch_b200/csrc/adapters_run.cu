// adapters_run.cu -- workspace sizes and launches of the adapters' forward and backward (adapters.cu:
// fp32 FMA kernels, adapters_tc.cu: tensor-core kernels).

namespace moe {

// Which forward: adapters_few_kernel for fp32, and for bf16 while its reads of A_a and W_r from L2 (which grow with
// m d (8 r + n)) cost less than the grouped tensor-core pass takes at least. Measured, few rows against tensor cores:
// 12 against 16 us for 512 rows (d 512, n 64, r 16), 29 against 20 for 2048; 13 against 24 for 128 rows of d 2048, 31
// against 25 for 512; 20 against 23 for 64 rows (d 1024, n 128, r 64), 27 against 23 for 128; 10 against 13 for 2048
// rows of d 64, 16 against 13 for 4096.
static bool adapters_few(int64_t m, int d, int n, int r, moe_dtype dt) {
    return dt == MOE_F32 || (m <= 2048 && m * d * (8 * r + n) <= (int64_t)1 << 26);
}

size_t router_adapters_workspace_bytes(int64_t m, int32_t d, int32_t n, int32_t r, int32_t na, moe_dtype dt) {
    if (m < 1 || d < 1 || n < 1 || n > kMaxExperts || r < 1 || r > kMaxRank || na < 1 || adapters_few(m, d, n, r, dt)) return 0;
    return atc_layout(m, d, n, r, na, nullptr, nullptr);
}

size_t router_adapters_grad_workspace_bytes(int64_t m, int32_t d, int32_t n, int32_t r, int32_t na, moe_dtype dt) {
    if (m < 1 || d < 1 || n < 1 || n > kMaxExperts || r < 1 || r > kMaxRank || na < 1) return 0;
    if (dt == MOE_BF16) return agt_layout(m, d, n, r, na, nullptr, nullptr);
    return adapter_ws_layout(m, d, n, r, na, nullptr, nullptr);
}

cudaError_t launch_router_adapters(const void* x, moe_dtype dt, const float* w_r, const void* a, const void* b,
                                   const int32_t* idx, const float* scale, int64_t m, int d, int n, int r, int na,
                                   float* logits, float* hidden, void* workspace, cudaStream_t stream) {
    if (m == 0) return cudaSuccess;
    if (dt == MOE_F32)
        return launch_adapters_few(static_cast<const float*>(x), w_r, static_cast<const float*>(a),
                                   static_cast<const float*>(b), idx, scale, m, d, n, r, na, logits, hidden, stream);
    const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16*>(x), *ab = static_cast<const __nv_bfloat16*>(a),
                        *bb = static_cast<const __nv_bfloat16*>(b);
    if (adapters_few(m, d, n, r, dt))
        return launch_adapters_few(xb, w_r, ab, bb, idx, scale, m, d, n, r, na, logits, hidden, stream);
    return launch_router_adapters_tc(xb, w_r, ab, bb, idx, scale, m, d, n, r, na, logits, hidden, workspace, stream);
}

static cudaError_t launch_adapters_grad_f32(const float* dh, const float* x, const float* w_r, const float* a,
                                            const float* b, const int32_t* idx, const float* scale,
                                            const float* hidden, int64_t m, int d, int n, int r, int na, float* dx,
                                            float* da, float* db, float* dw_r, void* workspace, cudaStream_t stream) {
    AdapterWs w;
    adapter_ws_layout(m, d, n, r, na, &w, static_cast<char*>(workspace));
    PrepExtra extra = {};
    extra.dh = dh; extra.b = b; extra.scale = scale; extra.n = n; extra.r = r; extra.du = w.du;
    cudaError_t e = launch_adapter_prep(idx, m, na, w.plan, nullptr, 0, extra, stream);
    if (e != cudaSuccess) return e;
    if (dx) {
        e = launch_pdl(adapters_dx_kernel, dim3((unsigned)((m + 15) / 16), (unsigned)((d + 127) / 128)),
                       dim3(adp::kThreads), 0, stream, dh, w_r, a, idx, w.du, m, d, n, r, na, dx);
        if (e != cudaSuccess) return e;
    }
    RowsTasks tasks = {};
    tasks.count = dw_r ? 3 : 2;
    const float *X[3] = {x, hidden, dh}, *Y[3] = {w.du, dh, x}, *S[3] = {nullptr, scale, nullptr};
    float* out[3] = {da, db, dw_r};
    int64_t blocks = 0, fold = 0;
    for (int i = 0; i < tasks.count; ++i) {
        RowsTask& t = tasks.t[i] = w.task[i];
        t.X = X[i]; t.Y = Y[i]; t.scale = S[i]; t.out = out[i];
        blocks += (int64_t)t.ptiles * t.qtiles * t.segs;
        fold += ((int64_t)t.np * t.nq + adp::kThreads - 1) / adp::kThreads;
    }
    e = launch_pdl(rows_outer_kernel, dim3((unsigned)blocks), dim3(adp::kThreads), 0, stream, tasks, m, na + 1, w.plan);
    if (e != cudaSuccess) return e;
    return launch_pdl(rows_fold_kernel, dim3((unsigned)fold, (unsigned)na), dim3(adp::kThreads), 0, stream, tasks, w.plan);
}

cudaError_t launch_router_adapters_grad(const float* dh, const void* x, moe_dtype dt, const float* w_r, const void* a,
                                        const void* b, const int32_t* idx, const float* scale, const float* hidden,
                                        int64_t m, int d, int n, int r, int na, void* dx, float* da, float* db,
                                        float* dw_r, void* workspace, cudaStream_t stream) {
    if (m == 0) {  // no rows: the sums are zero
        cudaError_t e = cudaMemsetAsync(da, 0, sizeof(float) * (size_t)na * r * d, stream);
        if (e == cudaSuccess) e = cudaMemsetAsync(db, 0, sizeof(float) * (size_t)na * n * r, stream);
        if (e == cudaSuccess && dw_r) e = cudaMemsetAsync(dw_r, 0, sizeof(float) * (size_t)d * n, stream);
        return e;
    }
    if (dt == MOE_BF16)
        return launch_adapters_grad_tc(dh, static_cast<const __nv_bfloat16*>(x), w_r,
                                       static_cast<const __nv_bfloat16*>(a), static_cast<const __nv_bfloat16*>(b), idx,
                                       scale, hidden, m, d, n, r, na, static_cast<__nv_bfloat16*>(dx), da, db, dw_r,
                                       workspace, stream);
    return launch_adapters_grad_f32(dh, static_cast<const float*>(x), w_r, static_cast<const float*>(a),
                                    static_cast<const float*>(b), idx, scale, hidden, m, d, n, r, na,
                                    static_cast<float*>(dx), da, db, dw_r, workspace, stream);
}

}  // namespace moe
