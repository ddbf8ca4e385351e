// ortho.cu -- orthogonalising a batch of weight updates by Newton-Schulz products.
//
// X = M / (|M| + eps) with the Frobenius norm, then steps of A = X X^T, B = b A + c A A, X = a X + B X: the
// singular vectors stay, the singular values go through the polynomial a s + b s^3 + c s^5 in every step. Two
// kernels make X (the squares' sums; the split into halves, with the transposition of a tall matrix), three
// a step are products (ortho_gemm.cuh). The first two move what they have to at the copy rate: 268 MB of bf16 42 us,
// the same into two halves 122.
#include <cmath>

#include "ortho_gemm.cuh"
#include "ortho_values.cuh"

namespace ep {

namespace {

constexpr int kSquareThreads = 512;
constexpr int kSquareParts = 64;       // CTAs that add up one matrix, at most
constexpr int64_t kSquarePart = 65536;  // values of each, at least

// The squares of `n` values times `scale`^2, this thread's part.
template <typename V>
__device__ __forceinline__ float squares(const V *p, int64_t n, float scale, bool &any) {
    constexpr int kVec = Io<V>::kVec;
    float acc[4] = {0, 0, 0, 0};
    const int64_t head = min(values_to_boundary(p), n);
    const auto one = [&](int64_t i) {
        const float v = Io<V>::load(p + i);
        any |= v != 0.0f;
        acc[0] = fmaf(v * scale, v * scale, acc[0]);
    };
    if (threadIdx.x < head) one(threadIdx.x);
    const uint4 *q = reinterpret_cast<const uint4 *>(p + head);
    const int64_t vecs = (n - head) / kVec;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vecs; i += kSquareThreads) {
        float v[kVec];
        Io<V>::unpack(q[i], v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            any |= v[j] != 0.0f;
            acc[j % 4] = fmaf(v[j] * scale, v[j] * scale, acc[j % 4]);
        }
    }
    const int64_t tail = head + vecs * kVec + threadIdx.x;
    if (tail < n) one(tail);
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// The sum over the CTA, in every thread.
__device__ float square_cta_sum(float v) {
    __shared__ float part[kSquareThreads / 32];
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = threadIdx.x % 32 < kSquareThreads / 32 ? part[threadIdx.x % 32] : 0.0f;
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// partial[CTA] = the sum of the squares of its part of a matrix. Where that leaves fp32's range, the values
// are read again, times a power of two.
template <typename V>
__global__ void __launch_bounds__(kSquareThreads) ortho_square_kernel(const V *m, int64_t size, int parts, double *partial) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t matrix = blockIdx.x / parts;
    const int part = blockIdx.x % parts;
    const int64_t begin = size * part / parts, end = size * (part + 1) / parts;
    const V *p = m + matrix * size + begin;
    bool any = false;
    float sum = square_cta_sum(squares(p, end - begin, 1.0f, any));
    any = __syncthreads_or(any);
    double back = 1.0;
    if (any && !(sum >= 0x1p-90f && sum <= 0x1p126f)) {
        const bool small = sum < 0x1p-90f;
        sum = square_cta_sum(squares(p, end - begin, small ? 0x1p90f : 0x1p-90f, any));
        back = small ? 0x1p-180 : 0x1p180;
    }
    if (threadIdx.x == 0) partial[blockIdx.x] = sum * back;
}

__device__ OrthoScale matrix_scale(const double *partial, int parts, float eps) {
    __shared__ OrthoScale shared;
    if (threadIdx.x < 32) {
        double v = 0;
        for (int i = threadIdx.x; i < parts; i += 32) v += partial[i];
        for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        if (threadIdx.x == 0) shared = ortho_scale(v, eps);
    }
    __syncthreads();
    return shared;
}

constexpr int kSplitThreads = 256;
constexpr int kSplitTile = 64;

// hi and lo of a matrix [N, K] whose rows stay rows: a thread takes 8 columns, zeros behind the last.
template <typename V>
__global__ void __launch_bounds__(kSplitThreads) ortho_split_kernel(const V *m, int rows, int cols, int pitch, int ctas, int parts,
                                                                    const double *partial, float eps, uint16_t *hi,
                                                                    uint16_t *lo) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t matrix = blockIdx.x / ctas;
    const OrthoScale scale = matrix_scale(partial + matrix * parts, parts, eps);
    const V *src = m + matrix * rows * cols;
    const int words = pitch / 8;
    const int64_t total = (int64_t)rows * words;
    const bool vector = cols % 8 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0;
    for (int64_t i = (int64_t)blockIdx.x % ctas * kSplitThreads + threadIdx.x; i < total; i += (int64_t)ctas * kSplitThreads) {
        const int64_t row = i / words;
        const int c = (int)(i % words) * 8;
        const V *p = src + row * cols + c;
        float v[8];
        if (vector) {
            constexpr int kVec = Io<V>::kVec;
#pragma unroll
            for (int j = 0; j < 8 / kVec; ++j) {
                float u[kVec];
                Io<V>::unpack(reinterpret_cast<const uint4 *>(p)[j], u);
#pragma unroll
                for (int k = 0; k < kVec; ++k) v[j * kVec + k] = u[k];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? Io<V>::load(p + j) : 0.0f;
        }
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split_pair(scale(v[2 * j]), scale(v[2 * j + 1]), h[j], l[j]);
        const size_t to = ((size_t)matrix * rows + row) * words + i % words;
        st_v4(reinterpret_cast<uint4 *>(hi) + to, make_uint4(h[0], h[1], h[2], h[3]));
        st_v4(reinterpret_cast<uint4 *>(lo) + to, make_uint4(l[0], l[1], l[2], l[3]));
    }
}

// The same for a matrix [N, K] that is held as [K, N]: tiles of 64 x 64 through shared memory.
template <typename V>
__global__ void __launch_bounds__(kSplitThreads) ortho_split_transposed_kernel(const V *m, int N, int K, int pitch, int ctas,
                                                                               int parts, const double *partial, float eps,
                                                                               uint16_t *hi, uint16_t *lo) {
    __shared__ float tile[kSplitTile][kSplitTile + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t matrix = blockIdx.x / ctas;
    const OrthoScale scale = matrix_scale(partial + matrix * parts, parts, eps);
    const V *src = m + matrix * N * K;
    const int across = (K + kSplitTile - 1) / kSplitTile;
    const int64_t tiles = (int64_t)across * ((N + kSplitTile - 1) / kSplitTile);
    for (int64_t t = blockIdx.x % ctas; t < tiles; t += ctas) {
        const int n0 = (int)(t / across) * kSplitTile, k0 = (int)(t % across) * kSplitTile;
        __syncthreads();
        for (int i = threadIdx.x; i < kSplitTile * kSplitTile; i += kSplitThreads) {
            const int r = i / kSplitTile, c = i % kSplitTile;
            tile[r][c] = n0 + r < N && k0 + c < K ? scale(Io<V>::load(src + (int64_t)(n0 + r) * K + k0 + c)) : 0.0f;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kSplitTile * kSplitTile / 8; i += kSplitThreads) {
            const int r = i / (kSplitTile / 8), c = i % (kSplitTile / 8) * 8;  // row k0 + r, from n0 + c on
            if (k0 + r >= K || n0 + c >= pitch) continue;
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split_pair(tile[c + 2 * j][r], tile[c + 2 * j + 1][r], h[j], l[j]);
            const size_t to = (((size_t)matrix * K + k0 + r) * pitch + n0 + c) / 8;
            st_v4(reinterpret_cast<uint4 *>(hi) + to, make_uint4(h[0], h[1], h[2], h[3]));
            st_v4(reinterpret_cast<uint4 *>(lo) + to, make_uint4(l[0], l[1], l[2], l[3]));
        }
    }
}

struct OrthoPlan {
    int m, n, mp, np, parts;
    bool tall;
    size_t partial, x[2], lo[2], a, b, da, db, bytes;  // offsets
};

OrthoPlan plan_of(const ep_ortho_config &c) {
    OrthoPlan p = {};
    p.tall = c.N > c.K;
    p.m = p.tall ? c.K : c.N;
    p.n = p.tall ? c.N : c.K;
    p.mp = (p.m + 7) / 8 * 8;
    p.np = (p.n + 7) / 8 * 8;
    const int64_t parts = ((int64_t)c.N * c.K + kSquarePart - 1) / kSquarePart;
    p.parts = (int)(parts < kSquareParts ? parts : kSquareParts);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t batch = (size_t)c.B, x = batch * p.m * p.np * 2, a = batch * p.m * p.mp * 2;
    p.partial = take(batch * p.parts * sizeof(double));
    for (int i = 0; i < 2; ++i) {  // both halves: a step's are read by all while the next one's are written
        p.x[i] = take(x);
        p.lo[i] = take(x);
    }
    p.a = take(a);
    p.b = take(a);
    p.da = take((batch * p.mp + 32) * sizeof(float));
    p.db = take((batch * p.mp + 32) * sizeof(float));
    p.bytes = at;
    return p;
}

template <typename V>
cudaError_t make_x(const ep_ortho_config &c, const OrthoPlan &q, const void *m, double *partial, uint16_t *hi, uint16_t *lo,
                   cudaStream_t s) {
    const V *src = static_cast<const V *>(m);
    const int sms = current_device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    cudaError_t e = launch_dependent(ortho_square_kernel<V>, dim3((unsigned)(c.B * q.parts)), dim3(kSquareThreads), 0, s, src,
                                     (int64_t)c.N * c.K, q.parts, partial);
    if (e != cudaSuccess) return e;
    // CTAs of a matrix: all of its work items, or as many as fill the GPU eight times over with the others'
    const int64_t items = q.tall ? (int64_t)((c.N + kSplitTile - 1) / kSplitTile) * ((c.K + kSplitTile - 1) / kSplitTile)
                                 : ((int64_t)q.m * (q.np / 8) + kSplitThreads - 1) / kSplitThreads;
    const int64_t most = ((int64_t)sms * 8 * 4 + c.B - 1) / c.B;
    const int ctas = (int)(items < most ? items : most);
    if (q.tall)
        return launch_dependent(ortho_split_transposed_kernel<V>, dim3((unsigned)(c.B * ctas)), dim3(kSplitThreads), 0, s, src, c.N,
                                c.K, q.np, ctas, q.parts, (const double *)partial, c.eps, hi, lo);
    return launch_dependent(ortho_split_kernel<V>, dim3((unsigned)(c.B * ctas)), dim3(kSplitThreads), 0, s, src, c.N, c.K, q.np,
                            ctas, q.parts, (const double *)partial, c.eps, hi, lo);
}

// What a product reads and writes, as tensors in global memory.
struct OrthoOperands {
    const uint16_t *a, *b, *b_lo;  // operands
    const uint16_t *in[2];       // what its epilogue reads beside them
    const uint16_t *out[2];      // what it writes; Apply's last step: the result
};

template <OrthoOp OP, int CG, int NB, bool SPLIT = false>
cudaError_t product(OrthoParams &p, const OrthoOperands &q, cudaStream_t s) {
    using Sh = OrthoShape<OP, CG, NB>;
    // the maps' type says bf16: all that depends on it is what fills the outside, zeros for both
    const int64_t x = OP == OrthoOp::kGram ? p.np : p.mp, wide = Sh::kSymmetric ? p.mp : p.np;
    bool ok = make_map(&p.a, q.a, 2, x, p.m, p.batch, kGemmBK, kGemmBM) &&
              (Sh::kBMn ? make_map(&p.b, q.b, 2, p.np, p.m, p.batch, 64, kGemmBK)
                        : make_map(&p.b, q.b, 2, x, p.m, p.batch, kGemmBK, Sh::kBRows));
    if (OP == OrthoOp::kApply && p.form == OrthoForm::kWhole) ok = ok && make_map(&p.b_lo, q.b_lo, 2, p.np, p.m, p.batch, 64, kGemmBK);
    for (int i = 0; i < 2; ++i) {
        if (q.in[i]) ok = ok && make_piece_map(&p.in[i], q.in[i], wide, p.m, p.batch);
        if (!q.out[i]) continue;
        if (!p.result)
            ok = ok && make_piece_map(&p.out[i], q.out[i], wide, p.m, p.batch);
        else if ((p.transposed ? p.m : p.n) % 8 == 0)  // else it is written value by value
            ok = ok && make_piece_map(&p.out[i], q.out[i], p.transposed ? p.m : p.n, p.transposed ? p.n : p.m, p.batch);
    }
    if (!ok) return cudaErrorInvalidValue;
    auto kernel = ortho_gemm_kernel<OP, CG, NB, SPLIT>;
    static SharedMemoryLimit limit;
    cudaError_t e = limit.allow(kernel, Sh::kSmem);
    if (e != cudaSuccess) return e;
    const int sms = current_device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t tiles = (int64_t)OrthoWalk<OP, CG, NB>::tiles(p.m, p.n) * p.batch;
    const int ctas = SPLIT ? p.split : CG;  // of a cluster
    const int64_t grid = tiles * ctas < sms ? tiles * ctas : sms / ctas * ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The tile of a product: by CTA pairs of 256 x 256 where those are more than the SMs' pairs, else the
// narrower one where that leaves fewer columns for the SM that has most (7 of 1000 x 360 145 -> 142 us, 5 of 384 x 1536
// 139 -> 134); a long contraction of few tiles is split over as many CTAs as leave
// each four stages of it (256 x 256 from 7168: 23 us by one CTA a tile).
template <OrthoOp OP>
cudaError_t choose(OrthoParams &p, const OrthoOperands &q, cudaStream_t s) {
    const int64_t sms = current_device_sm_count();
    if ((int64_t)OrthoWalk<OP, 2, 256>::tiles(p.m, p.n) * p.batch * 2 > sms) return product<OP, 2, 256>(p, q, s);
    const int64_t narrow = (int64_t)OrthoWalk<OP, 1, 64>::tiles(p.m, p.n) * p.batch;
    if constexpr (OP == OrthoOp::kGram) {
        const int64_t stages = (p.n + kGemmBK - 1) / kGemmBK;
        for (p.split = 8; p.split > 1; p.split /= 2)
            if (narrow * p.split <= sms && stages >= 4 * p.split) return product<OP, 1, 64, true>(p, q, s);
    }
    const int64_t wide = (int64_t)OrthoWalk<OP, 1, 128>::tiles(p.m, p.n) * p.batch;
    if ((narrow + sms - 1) / sms < 2 * ((wide + sms - 1) / sms)) return product<OP, 1, 64>(p, q, s);
    return product<OP, 1, 128>(p, q, s);
}

}  // namespace

size_t ortho_workspace_bytes(const ep_ortho_config &c) { return ortho_fits_any_device(c) ? 256 : plan_of(c).bytes; }

bool ortho_steps(const float *k, int32_t steps, int32_t rows, OrthoForm *form) {
    double s = 1.0, alike = 1.0 / std::sqrt((double)rows);  // the largest singular value; all of them, if they are alike
    for (int i = 0; i < steps; ++i) {
        double growth = 1.0;  // by the later steps, of what X has none of
        for (int j = i + 1; j < steps; ++j) growth *= std::fabs((double)k[3 * j]);
        const double a = k[3 * i], b = k[3 * i + 1], c = k[3 * i + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        const double t = s * s;  // squares of singular values: [0, t]
        const auto poly = [&](double u) { return std::fabs(b * u + c * u * u); };
        double most = poly(t);
        if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < t) most = std::fmax(most, poly(-b / (2 * c)));
        if (!(most < 31)) return false;
        const auto value = [&](double u) { return std::fabs(a + b * u + c * u * u) * std::sqrt(u); };
        double next = value(t);
        // where the derivative a + 3 b u + 5 c u^2 vanishes
        double roots[2] = {-1, -1};
        if (c != 0) {
            const double disc = 9 * b * b - 20 * a * c;
            if (disc >= 0) roots[0] = (-3 * b - std::sqrt(disc)) / (10 * c), roots[1] = (-3 * b + std::sqrt(disc)) / (10 * c);
        } else if (b != 0) {
            roots[0] = -a / (3 * b);
        }
        for (const double u : roots)
            if (u > 0 && u < t) next = std::fmax(next, value(u));
        if (form) {
            // kDiagonal: what it leaves is within 2^-12 `most` times X, and grows to 10 times 2^-12 X at most (the last two of
            // the default steps; at 30, the last three, 64 x 256 of rank 16 is 0.19% off after five steps instead of 0.10).
            // kUpper: B is about a third of a at most, so that 2^-12 B is little beside what A's and B's roundings leave (five
            // steps of 256 x 384, the first two, free; the third as well would be 0.085% off instead of 0.067).
            form[i] = most * growth <= 10                          ? OrthoForm::kDiagonal
                      : poly(alike * alike) <= std::fabs(a) * 0.35 ? OrthoForm::kUpper
                                                                   : OrthoForm::kWhole;
        }
        s = next * 1.01;  // and roundings
        alike = std::fmin(value(alike * alike), s);
        if (!(s < 4)) return false;
    }
    return true;
}

bool ortho_fits(const float *k, int32_t steps) { return ortho_steps(k, steps, 1, nullptr); }

cudaError_t launch_orthogonalize(const ep_ortho_config &c, const float *k, const void *m, ep_bf16 *out, void *workspace,
                                 cudaStream_t s) {
    cudaError_t e;
    if (ortho_fits_fused(c)) {
        bool ran = false;
        e = launch_ortho_fused(c, k, m, out, &ran, s);
        if (e != cudaSuccess || ran) return e;
    }
    const OrthoPlan q = plan_of(c);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const auto half = [&](size_t at) { return reinterpret_cast<uint16_t *>(ws + at); };
    uint16_t *x[2] = {half(q.x[0]), half(q.x[1])}, *lo[2] = {half(q.lo[0]), half(q.lo[1])}, *a = half(q.a), *b = half(q.b);
    float *da = reinterpret_cast<float *>(ws + q.da), *db = reinterpret_cast<float *>(ws + q.db);
    double *partial = reinterpret_cast<double *>(ws + q.partial);
    e = c.dtype == EP_F32    ? make_x<float>(c, q, m, partial, x[0], lo[0], s)
        : c.dtype == EP_BF16 ? make_x<__nv_bfloat16>(c, q, m, partial, x[0], lo[0], s)
                             : make_x<__half>(c, q, m, partial, x[0], lo[0], s);
    if (e != cudaSuccess) return e;
    OrthoParams p = {};
    e = expert_error_word(&p.error);
    if (e != cudaSuccess) return e;
    p.batch = c.B;
    p.m = q.m;
    p.n = q.n;
    p.mp = q.mp;
    p.np = q.np;
    p.transposed = q.tall;
    OrthoForm form[64];
    ortho_steps(k, c.steps, q.m, form);
    for (int i = 0; i < c.steps; ++i) {
        const uint16_t *now = x[i % 2], *now_lo = lo[i % 2];
        p.ca = k[3 * i], p.cb = k[3 * i + 1], p.cc = k[3 * i + 2];
        p.d_out = da;
        p.split_out = a;
        e = choose<OrthoOp::kGram>(p, {now, now, nullptr, {}, {a}}, s);
        if (e != cudaSuccess) return e;
        p.d = da;
        p.d_out = db;
        e = choose<OrthoOp::kPoly>(p, {a, a, nullptr, {a}, {b}}, s);
        if (e != cudaSuccess) return e;
        p.d = db;
        const bool last = i + 1 == c.steps;
        p.result = last ? out : nullptr;
        p.form = form[i];
        e = choose<OrthoOp::kApply>(p, {b, now, now_lo, {now, now_lo}, {last ? out : x[(i + 1) % 2], last ? nullptr : lo[(i + 1) % 2]}}, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ep
