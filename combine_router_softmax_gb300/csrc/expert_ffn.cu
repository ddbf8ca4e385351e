// expert_ffn.cu -- launchers of the experts' gated block, forward and backward
// (the kernel: expert_gemm.cuh).
#include "expert_gemm.cuh"
#include "expert_stream.cuh"

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

}  // namespace

namespace {

bool encode_map(CUtensorMap *m, const void *base, int bytes, int64_t x, int64_t y, int64_t z, int bx, int by,
                CUtensorMapSwizzle swizzle) {
    EncodeTiled encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
    const cuuint64_t strides[2] = {(cuuint64_t)x * bytes, (cuuint64_t)x * (cuuint64_t)y * bytes};
    const cuuint32_t box[3] = {(cuuint32_t)bx, (cuuint32_t)by, 1}, ones[3] = {1, 1, 1};
    return encode(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, z > 0 ? 3 : 2,
                  const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_map(CUtensorMap *m, const void *base, int bytes, int64_t x, int64_t y, int64_t z, int bx, int by) {
    return encode_map(m, base, bytes, x, y, z, bx, by, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool make_piece_map(CUtensorMap *m, const void *base, int64_t x, int64_t y, int64_t z) {
    return encode_map(m, base, 2, x, y, z, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

namespace {

// A operand of a row product: rows x k.
bool rows_map(GemmParams &p, int i, const ep_bf16 *base, int64_t k) {
    return make_map(&p.a[i], base, 2, k, p.S, 0, kGemmBK, 128) && make_map(&p.a64[i], base, 2, k, p.S, 0, kGemmBK, 64) &&
           make_map(&p.a16[i], base, 2, k, p.S, 0, kGemmBK, 16);
}

template <ExpertOp OP, int CG, int NB>
cudaError_t launch(GemmParams &p, int64_t most_tiles, cudaStream_t s) {
    using Sh = GemmShape<OP, CG, NB>;
    auto kernel = expert_gemm_kernel<OP, CG, NB>;
    cudaError_t e = expert_error_word(&p.error);
    if (e != cudaSuccess) return e;
    const size_t smem = Sh::smem_bytes(p.E);
    static SharedMemoryLimit limit;
    e = limit.allow(kernel, smem);
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
    p.saved_bf16 = c.saved_bf16;
    return p;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of bm rows, at most: every expert that has rows can end inside one.
int64_t row_tiles(const GemmParams &p, int bm) { return p.S / bm + (p.E < p.S ? p.E : p.S); }

// Which tile a product takes: the narrowest whose tiles are all resident at once, as a narrower one
// gives each SM less and ends sooner (8 experts x 128 rows, 2048 to 1024 and back, forward: 64 wide
// 31 us, 128 wide 27, 256 wide 33; at half the experts 17, 18, 26; at twice the experts 56, 47, 48). With
// more tiles than SMs, 256 wide, and by CTA pairs of 256 rows where an expert has more than
// `pair_rows`: a pair halves what each SM reads of the weights (16 experts, 2048 to 1024 and back,
// forward: 200 rows each 60 us single, 57 pairs; 512 rows 100 and 86).
enum class TileShape { k64, k128, k256, kPair };
template <typename Tiles>
TileShape choose(const GemmParams &p, int pair_rows, Tiles tiles) {
    const int64_t sms = current_device_sm_count();
    if (tiles(64) <= sms) return TileShape::k64;
    if (tiles(128) <= sms) return TileShape::k128;
    return tiles(256) > sms && p.S > (int64_t)pair_rows * p.E ? TileShape::kPair : TileShape::k256;
}

// Few rows: the weights are streamed past the rows' registers (expert_stream.cuh), 5% faster than tiles
// (8 experts with one row each, 4096 to 1024: 39 us against 41). Up to as many rows as one pass takes;
// with more, an expert that has most of them would be streamed again and again.
bool streams(const ep_ffn_config &c) { return c.rows <= kStreamTokens; }

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
        constexpr int kBoxN = OP == ExpertOp::kGateUp ? Sh::kGate : Sh::kBRows;
        const bool ok = Sh::kBMn ? make_map(&p.b[i], r.b[i], 2, p.N[0], p.K, p.E, 64, kGemmBK)
                                 : make_map(&p.b[i], r.b[i], 2, p.K, p.N[0], p.E, kGemmBK, kBoxN);
        if (!ok) return cudaErrorInvalidValue;
    }
    return launch<OP, CG, NB>(p, row_tiles(p, kGemmBM * CG) * ceil_div(p.N[0], Sh::kOutN), s);
}

template <ExpertOp OP>
cudaError_t row_product(GemmParams &p, const RowProduct &r, cudaStream_t s) {
    constexpr int kPerColumn = 256 / GemmShape<OP, 1, 256>::kOutN;  // accumulator columns of an output column
    const int64_t m = p.S / kGemmBM > p.E ? p.S / kGemmBM : p.E < p.S ? p.E : p.S;
    switch (choose(p, kGemmBM, [&](int width) { return m * ceil_div((int64_t)p.N[0] * kPerColumn, width); })) {
        case TileShape::k64: return run_rows<OP, 1, 64>(p, r, s);
        case TileShape::k128: return run_rows<OP, 1, 128>(p, r, s);
        case TileShape::k256: return run_rows<OP, 1, 256>(p, r, s);
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
                              const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, uint16_t *g,
                              uint16_t *u, ep_bf16 *h, ep_bf16 *y, cudaStream_t s) {
    if (!g && streams(c)) {
        StreamParams q = {};
        q.x = rows;
        q.expert_offset = expert_offset;
        q.y = h;
        q.S = c.rows;
        q.N = c.I;
        q.K = c.H;
        q.E = c.E;
        const cudaError_t e = launch_stream<true, 0>(q, w_gate, w_up, s);
        if (e != cudaSuccess) return e;
        q.x = h;
        q.y = y;
        q.N = c.H;
        q.K = c.I;
        return launch_stream<false, 0>(q, w_down, nullptr, s);
    }
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
                                       const uint16_t *g, const uint16_t *u, const ep_bf16 *h, const ep_bf16 *d_y,
                                       ep_bf16 *d_g, ep_bf16 *d_u, ep_bf16 *d_rows, ep_bf16 *d_w_gate,
                                       ep_bf16 *d_w_up, ep_bf16 *d_w_down, cudaStream_t s) {
    GemmParams p = base_params(c, expert_offset);
    p.K = c.H;
    p.N[0] = c.I;
    p.out[0] = d_g;
    p.out[1] = d_u;
    p.g = const_cast<uint16_t *>(g);
    p.u = const_cast<uint16_t *>(u);
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
        if (!make_map(&p.a[i], w.a, 2, w.M, p.S, 0, 64, kGemmBK) || !make_map(&p.b[i], w.b, 2, w.N, p.S, 0, 64, kGemmBK))
            return cudaErrorInvalidValue;
    }
    if (p.problems == 0) return cudaSuccess;
    // the epilogue is a large part of these tiles: between 64 and 256 wide there is nothing to gain, and
    // pairs, which share it less evenly, pay later (2048 x 1024, 16 experts: 256 rows each 65 us single,
    // 91 pairs; 512 rows 101 and 97)
    switch (choose(p, 3 * kGemmBM, [&](int width) { return weight_tiles(p, kGemmBM, width < 128 ? 64 : 256); })) {
        case TileShape::k64: return launch<ExpertOp::kDWeight, 1, 64>(p, weight_tiles(p, kGemmBM, 64), s);
        case TileShape::kPair: return launch<ExpertOp::kDWeight, 2, 256>(p, weight_tiles(p, 2 * kGemmBM, 256), s);
        default: return launch<ExpertOp::kDWeight, 1, 256>(p, weight_tiles(p, kGemmBM, 256), s);
    }
}

}  // namespace ep
