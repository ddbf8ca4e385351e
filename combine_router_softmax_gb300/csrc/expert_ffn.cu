// expert_ffn.cu -- launchers of the experts' gated block, forward and backward
// (the kernel: expert_gemm.cuh).
#include "expert_gemm.cuh"

namespace ep {

namespace {

__device__ int32_t g_expert_error;

}  // namespace

cudaError_t expert_error_word(int32_t **addr) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(addr), g_expert_error);
}

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// A bf16 matrix [y][x], or [z][y][x], read in boxes of bx by by elements, 128-byte swizzled.
// What lies outside reads as zero.
bool make_map(CUtensorMap *m, const ep_bf16 *base, int64_t x, int64_t y, int64_t z, int bx, int by) {
    EncodeTiled encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)x * 2, (cuuint64_t)x * (cuuint64_t)y * 2};
    const cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, 1}, ones[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, z > 0 ? 3 : 2, const_cast<ep_bf16 *>(base), dims, strides, box,
                  ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A operand of a row product: rows x k.
bool rows_map(GemmParams &p, int i, const ep_bf16 *base, int64_t k) {
    return make_map(&p.a[i], base, k, p.S, 0, kGemmBK, kGemmBM) && make_map(&p.a16[i], base, k, p.S, 0, kGemmBK, 16);
}

template <ExpertOp OP, int CG, int NB>
cudaError_t launch(GemmParams &p, int64_t most_tiles, cudaStream_t s) {
    using Sh = GemmShape<OP, CG, NB>;
    auto kernel = expert_gemm_kernel<OP, CG, NB>;
    cudaError_t e = expert_error_word(&p.error);
    if (e != cudaSuccess) return e;
    const size_t smem = Sh::smem_bytes(p.E);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int sms = current_device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    int64_t grid = most_tiles * CG < sms ? most_tiles * CG : sms / CG * CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// An upper bound of a row product's tiles: every expert can end inside one.
int64_t row_tiles(const GemmParams &p, int bm, int out_n) {
    const int64_t m = (int64_t)p.S / bm + (p.E < p.S ? p.E : p.S);
    return m * ((p.N[0] + out_n - 1) / out_n);
}

GemmParams base_params(const ep_ffn_config &c, const int32_t *expert_offset) {
    GemmParams p = {};
    p.expert_offset = expert_offset;
    p.E = c.E;
    p.S = c.rows;
    return p;
}

template <int CG, int NB>
cudaError_t run_forward(const ep_ffn_config &c, const ep_bf16 *rows, const int32_t *expert_offset,
                              const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, ep_bf16 *g,
                        ep_bf16 *u, ep_bf16 *h, ep_bf16 *y, cudaStream_t s) {
    GemmParams p = base_params(c, expert_offset);
    p.K = c.H;
    p.N[0] = c.I;
    p.out[0] = h;
    p.g = g;
    p.u = u;
    if (!rows_map(p, 0, rows, c.H) || !make_map(&p.b[0], w_gate, c.H, c.I, c.E, kGemmBK, NB / 2) ||
        !make_map(&p.b[1], w_up, c.H, c.I, c.E, kGemmBK, NB / 2))
        return cudaErrorInvalidValue;
    cudaError_t e = launch<ExpertOp::kGateUp, CG, NB>(p, row_tiles(p, kGemmBM * CG, NB / 2), s);
    if (e != cudaSuccess) return e;

    p = base_params(c, expert_offset);
    p.K = c.I;
    p.N[0] = c.H;
    p.out[0] = y;
    if (!rows_map(p, 0, h, c.I) || !make_map(&p.b[0], w_down, c.I, c.H, c.E, kGemmBK, NB / CG)) return cudaErrorInvalidValue;
    return launch<ExpertOp::kDown, CG, NB>(p, row_tiles(p, kGemmBM * CG, NB), s);
}

template <int CG, int NB>
cudaError_t run_backward(const ep_ffn_config &c, const ep_bf16 *rows, const int32_t *expert_offset,
                                       const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down,
                                       const ep_bf16 *g, const ep_bf16 *u, const ep_bf16 *h, const ep_bf16 *d_y,
                                       ep_bf16 *d_g, ep_bf16 *d_u, ep_bf16 *d_rows, ep_bf16 *d_w_gate,
                         ep_bf16 *d_w_up, ep_bf16 *d_w_down, cudaStream_t s) {
    GemmParams p = base_params(c, expert_offset);
    p.K = c.H;
    p.N[0] = c.I;
    p.out[0] = d_g;
    p.out[1] = d_u;
    p.g = const_cast<ep_bf16 *>(g);
    p.u = const_cast<ep_bf16 *>(u);
    if (!rows_map(p, 0, d_y, c.H) || !make_map(&p.b[0], w_down, c.I, c.H, c.E, 64, kGemmBK)) return cudaErrorInvalidValue;
    cudaError_t e = launch<ExpertOp::kDGateUp, CG, NB>(p, row_tiles(p, kGemmBM * CG, NB), s);
    if (e != cudaSuccess) return e;

    if (d_rows) {
        p = base_params(c, expert_offset);
        p.K = c.I;
        p.N[0] = c.H;
        p.out[0] = d_rows;
        if (!rows_map(p, 0, d_g, c.I) || !rows_map(p, 1, d_u, c.I) ||
            !make_map(&p.b[0], w_gate, c.H, c.I, c.E, 64, kGemmBK) || !make_map(&p.b[1], w_up, c.H, c.I, c.E, 64, kGemmBK))
            return cudaErrorInvalidValue;
        e = launch<ExpertOp::kDRows, CG, NB>(p, row_tiles(p, kGemmBM * CG, NB), s);
        if (e != cudaSuccess) return e;
    }

    p = base_params(c, expert_offset);
    const struct {
        const ep_bf16 *a, *b;
        int32_t M, N;
        ep_bf16 *out;
    } want[3] = {{d_y, h, c.H, c.I, d_w_down}, {d_g, rows, c.I, c.H, d_w_gate}, {d_u, rows, c.I, c.H, d_w_up}};
    int64_t tiles = 0;
    for (const auto &w : want) {
        if (!w.out) continue;
        const int i = p.problems++;
        p.M[i] = w.M;
        p.N[i] = w.N;
        p.out[i] = w.out;
        if (!make_map(&p.a[i], w.a, w.M, p.S, 0, 64, kGemmBK) || !make_map(&p.b[i], w.b, w.N, p.S, 0, 64, kGemmBK))
            return cudaErrorInvalidValue;
        tiles += (int64_t)c.E * ((w.M + kGemmBM * CG - 1) / (kGemmBM * CG)) * ((w.N + NB - 1) / NB);
    }
    return p.problems ? launch<ExpertOp::kDWeight, CG, NB>(p, tiles, s) : cudaSuccess;
}

// A CTA pair takes tiles of 256 rows: worth it once an expert has more than one tile of 128.
bool pairs(const ep_ffn_config &c) { return c.rows > (int64_t)kGemmBM * c.E; }

}  // namespace

cudaError_t launch_expert_ffn(const ep_ffn_config &c, const ep_bf16 *rows, const int32_t *expert_offset,
                              const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, ep_bf16 *g,
                              ep_bf16 *u, ep_bf16 *h, ep_bf16 *y, cudaStream_t s) {
    const auto run = pairs(c) ? run_forward<2, 256> : run_forward<1, 256>;
    return run(c, rows, expert_offset, w_gate, w_up, w_down, g, u, h, y, s);
}

cudaError_t launch_expert_ffn_backward(const ep_ffn_config &c, const ep_bf16 *rows, const int32_t *expert_offset,
                                       const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down,
                                       const ep_bf16 *g, const ep_bf16 *u, const ep_bf16 *h, const ep_bf16 *d_y,
                                       ep_bf16 *d_g, ep_bf16 *d_u, ep_bf16 *d_rows, ep_bf16 *d_w_gate,
                                       ep_bf16 *d_w_up, ep_bf16 *d_w_down, cudaStream_t s) {
    const auto run = pairs(c) ? run_backward<2, 256> : run_backward<1, 256>;
    return run(c, rows, expert_offset, w_gate, w_up, w_down, g, u, h, d_y, d_g, d_u, d_rows, d_w_gate, d_w_up, d_w_down, s);
}

}  // namespace ep
