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
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

GemmParams base_params(const ep_ffn_config &c, const int32_t *expert_offset) {
    GemmParams p = {};
    p.expert_offset = expert_offset;
    p.E = c.E;
    p.S = c.rows;
    return p;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of bm rows, at most: every expert that has rows can end inside one.
int64_t row_tiles(const GemmParams &p, int bm) { return p.S / bm + (p.E < p.S ? p.E : p.S); }

// Which tile a product takes. Few tiles leave SMs idle and make each one's epilogue a large part of
// the whole, so below two tiles of 128 x 256 an SM they are 64 wide; with more than 128 rows an
// expert a CTA pair takes 256 rows at once, which halves what each SM reads of the weights.
enum class TileShape { kNarrow, kWide, kPair };
TileShape choose(const GemmParams &p, int64_t wide_tiles) {
    if (wide_tiles < 2 * (int64_t)current_device_sm_count()) return TileShape::kNarrow;
    return p.S > (int64_t)kGemmBM * p.E ? TileShape::kPair : TileShape::kWide;
}

// rows x k of the row product's A: halves [0, n) of it.
struct RowProduct {
    const ep_bf16 *a[2], *b[2];
};

template <ExpertOp OP, int CG, int NB>
cudaError_t run_rows(GemmParams &p, const RowProduct &r, cudaStream_t s) {
    using Sh = GemmShape<OP, CG, NB>;
    for (int i = 0; i < 2; ++i) {
        if (r.a[i] && !rows_map(p, i, r.a[i], p.K)) return cudaErrorInvalidValue;
        if (!r.b[i]) continue;
        // weights [E, N, K], or [E, K, N] where the product contracts their rows
        constexpr int kBoxN = OP == ExpertOp::kGateUp ? NB / 2 : Sh::kBRows;
        const bool ok = Sh::kBMn ? make_map(&p.b[i], r.b[i], p.N[0], p.K, p.E, 64, kGemmBK)
                                 : make_map(&p.b[i], r.b[i], p.K, p.N[0], p.E, kGemmBK, kBoxN);
        if (!ok) return cudaErrorInvalidValue;
    }
    return launch<OP, CG, NB>(p, row_tiles(p, kGemmBM * CG) * ceil_div(p.N[0], Sh::kOutN), s);
}

template <ExpertOp OP>
cudaError_t row_product(GemmParams &p, const RowProduct &r, cudaStream_t s) {
    const int64_t n = ceil_div(p.N[0], GemmShape<OP, 1, 256>::kOutN);
    const int64_t m = p.S / kGemmBM > p.E ? p.S / kGemmBM : p.E < p.S ? p.E : p.S;
    switch (choose(p, m * n)) {
        case TileShape::kNarrow: return run_rows<OP, 1, 64>(p, r, s);
        case TileShape::kWide: return run_rows<OP, 1, 256>(p, r, s);
        default: return run_rows<OP, 2, 256>(p, r, s);
    }
}

int64_t weight_tiles(const GemmParams &p, int bm, int bn) {
    int64_t n = 0;
    for (int i = 0; i < p.problems; ++i) n += ceil_div(p.M[i], bm) * ceil_div(p.N[i], bn);
    return n * p.E;
}

}  // namespace

cudaError_t launch_expert_ffn(const ep_ffn_config &c, const ep_bf16 *rows, const int32_t *expert_offset,
                              const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, ep_bf16 *g,
                              ep_bf16 *u, ep_bf16 *h, ep_bf16 *y, cudaStream_t s) {
    GemmParams p = base_params(c, expert_offset);
    p.K = c.H;
    p.N[0] = c.I;
    p.out[0] = h;
    p.g = g;
    p.u = u;
    const cudaError_t e = row_product<ExpertOp::kGateUp>(p, {{rows}, {w_gate, w_up}}, s);
    if (e != cudaSuccess) return e;
    p = base_params(c, expert_offset);
    p.K = c.I;
    p.N[0] = c.H;
    p.out[0] = y;
    return row_product<ExpertOp::kDown>(p, {{h}, {w_down}}, s);
}

cudaError_t launch_expert_ffn_backward(const ep_ffn_config &c, const ep_bf16 *rows, const int32_t *expert_offset,
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
    cudaError_t e = row_product<ExpertOp::kDGateUp>(p, {{d_y}, {w_down}}, s);
    if (e != cudaSuccess) return e;

    if (d_rows) {
        p = base_params(c, expert_offset);
        p.K = c.I;
        p.N[0] = c.H;
        p.out[0] = d_rows;
        e = row_product<ExpertOp::kDRows>(p, {{d_g, d_u}, {w_gate, w_up}}, s);
        if (e != cudaSuccess) return e;
    }

    p = base_params(c, expert_offset);
    const struct {
        const ep_bf16 *a, *b;
        int32_t M, N;
        ep_bf16 *out;
    } want[3] = {{d_y, h, c.H, c.I, d_w_down}, {d_g, rows, c.I, c.H, d_w_gate}, {d_u, rows, c.I, c.H, d_w_up}};
    for (const auto &w : want) {
        if (!w.out) continue;
        const int i = p.problems++;
        p.M[i] = w.M;
        p.N[i] = w.N;
        p.out[i] = w.out;
        if (!make_map(&p.a[i], w.a, w.M, p.S, 0, 64, kGemmBK) || !make_map(&p.b[i], w.b, w.N, p.S, 0, 64, kGemmBK))
            return cudaErrorInvalidValue;
    }
    if (p.problems == 0) return cudaSuccess;
    switch (choose(p, weight_tiles(p, kGemmBM, 256))) {
        case TileShape::kNarrow: return launch<ExpertOp::kDWeight, 1, 64>(p, weight_tiles(p, kGemmBM, 64), s);
        case TileShape::kWide: return launch<ExpertOp::kDWeight, 1, 256>(p, weight_tiles(p, kGemmBM, 256), s);
        default: return launch<ExpertOp::kDWeight, 2, 256>(p, weight_tiles(p, 2 * kGemmBM, 256), s);
    }
}

}  // namespace ep
