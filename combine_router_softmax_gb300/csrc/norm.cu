// norm.cu -- the norms before and after a block, fused with its gate and the residual scale.
//
// A row of H values is held in registers by a group of threads, a warp or a whole CTA: it is read
// once, its mean squares are sums over the group, and it is written once. HBM bounds it from a
// few hundred rows on, the launch and one chain of load, sum, store below.
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kNormWarps = 8;        // rows of a CTA where a row is one warp's
constexpr int kNormMaxPartials = 304;  // CTAs of the backward pass, at most: rows of partial sums

struct NormArgs {
    const void *x;
    const uint4 *y, *w_post, *w_next;
    const void *gate;
    void *out;
    uint4 *n;
    float *rstd_post, *rstd_next;  // forward: written where given; backward: read
    const void *d_out;
    const uint4 *d_n;
    void *d_x, *d_gate;
    uint4 *d_y;
    float *partial;  // [CTA][sums][H]
    int32_t T, vecs, kind, sigmoid;
    int32_t next_at, y_at;  // where a row of partial sums holds them, in H; -1: not wanted
    float eps, scale, offset, inv_h;
};

__device__ __forceinline__ void unpack8(const uint4 &q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight values of the residual stream, bf16 or float: `at` counts in eights.
template <bool F32>
struct Stream8 {
    uint4 q[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, size_t at) {
        const uint4 *s = static_cast<const uint4 *>(p) + at * (F32 ? 2 : 1);
        q[0] = *s;
        if constexpr (F32) q[1] = s[1];
    }
    __device__ __forceinline__ void clear() {
        q[0] = make_uint4(0, 0, 0, 0);
        if constexpr (F32) q[1] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(q[i].x), v[4 * i + 1] = __uint_as_float(q[i].y);
                v[4 * i + 2] = __uint_as_float(q[i].z), v[4 * i + 3] = __uint_as_float(q[i].w);
            }
        } else {
            unpack8(q[0], v);
        }
    }
    __device__ __forceinline__ static void store(void *p, size_t at, const float (&v)[8]) {
        uint4 *d = static_cast<uint4 *>(p) + at * (F32 ? 2 : 1);
        if constexpr (F32) {
            st_v4(d, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
            st_v4(d + 1, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
        } else {
            st_v4(d, pack8(v));
        }
    }
};

// The gate's factor and its derivative. With q = exp(-|g|) neither cancels at either end.
__device__ __forceinline__ float gate_act(float g, bool sigmoid) {
    if (!sigmoid) return g;
    const float q = __expf(-fabsf(g)), a = __fdividef(1.0f, 1.0f + q);
    return g >= 0.0f ? a : q * a;
}
__device__ __forceinline__ float gate_act(float g, bool sigmoid, float &slope) {
    if (!sigmoid) {
        slope = 1.0f;
        return g;
    }
    const float q = __expf(-fabsf(g)), a = __fdividef(1.0f, 1.0f + q);
    slope = q * a * a;
    return g >= 0.0f ? a : q * a;
}

// The sums of two values over the group, in every thread of it. `scratch`: not that of the sum before
// this one, which slower warps may still read.
template <bool WARP>
__device__ __forceinline__ void group_sum(float &a, float &b, float (*scratch)[32]) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, d);
    }
    if constexpr (!WARP) {
        const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
        if (lane == 0) scratch[0][threadIdx.x / 32] = a, scratch[1][threadIdx.x / 32] = b;
        __syncthreads();
        a = lane < warps ? scratch[0][lane] : 0.0f;
        b = lane < warps ? scratch[1][lane] : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
            b += __shfl_xor_sync(0xFFFFFFFFu, b, d);
        }
    }
}
template <bool WARP>
__device__ __forceinline__ void group_sum(float &a, float (*scratch)[32]) {
    float none = 0.0f;
    group_sum<WARP>(a, none, scratch);
}

// The thread's place: which row its group takes first, the step to the next, and its vectors
// i * stride + first of a row.
template <bool WARP>
struct Place {
    int first, stride, row, step;
    __device__ Place() {
        first = WARP ? threadIdx.x % 32 : threadIdx.x;
        stride = WARP ? 32 : blockDim.x;
        row = WARP ? blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
        step = WARP ? gridDim.x * (blockDim.x / 32) : gridDim.x;
    }
};

template <bool F32, bool WARP, int NV>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarps : 1024) block_norm_kernel(const NormArgs p) {
    __shared__ float scratch[2][2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const Place<WARP> at;
    const int t = at.row;
    if (WARP && t >= p.T) return;
    const size_t row = (size_t)t * p.vecs;
    Stream8<F32> x[NV];
    uint4 y[NV], wp[NV], wn[NV], g[NV];
    const bool has_y = p.y != nullptr, post = p.w_post != nullptr, next = p.n != nullptr;
    const float token_gate = p.kind == EP_GATE_TOKEN ? static_cast<const float *>(p.gate)[t] : 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * at.stride + at.first;
        const bool in = v < p.vecs;
        x[i].clear();
        y[i] = wp[i] = wn[i] = g[i] = make_uint4(0, 0, 0, 0);
        if (!in) continue;
        x[i].load(p.x, row + v);
        if (has_y) y[i] = p.y[row + v];
        if (post) wp[i] = p.w_post[v];
        if (next) wn[i] = p.w_next[v];
        if (p.kind == EP_GATE_CHANNEL) g[i] = static_cast<const uint4 *>(p.gate)[v];
        if (p.kind == EP_GATE_ELEMENT) g[i] = static_cast<const uint4 *>(p.gate)[row + v];
    }
    float r_y = 1.0f;
    if (post) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[8];
            unpack8(y[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
        }
        group_sum<WARP>(s, scratch[0]);
        r_y = rsqrtf(fmaf(s, p.inv_h, p.eps));
        if (p.rstd_post && at.first == 0) p.rstd_post[t] = r_y;
    }
    float out[NV][8], s = 0.0f;
    const float scale = p.kind == EP_GATE_TOKEN ? p.scale * gate_act(token_gate, p.sigmoid) : p.scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        x[i].get(out[i]);
        const int v = i * at.stride + at.first;
        if (v >= p.vecs) continue;
        if (has_y) {
            float z[8], w[8], a[8];
            unpack8(y[i], z);
            unpack8(wp[i], w);
            unpack8(g[i], a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (post) z[j] = (p.offset + w[j]) * (z[j] * r_y);
                const float f = p.kind == EP_GATE_CHANNEL || p.kind == EP_GATE_ELEMENT ? scale * gate_act(a[j], p.sigmoid) : scale;
                out[i][j] = fmaf(f, z[j], out[i][j]);
            }
            Stream8<F32>::store(p.out, row + v, out[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(out[i][j], out[i][j], s);
    }
    if (!next) return;
    group_sum<WARP>(s, scratch[1]);
    const float r = rsqrtf(fmaf(s, p.inv_h, p.eps));
    if (p.rstd_next && at.first == 0) p.rstd_next[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * at.stride + at.first;
        if (v >= p.vecs) continue;
        float w[8];
        unpack8(wn[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = (p.offset + w[j]) * (out[i][j] * r);
        st_v4(p.n + row + v, pack8(w));
    }
}

// The sums over rows that the backward pass keeps, a value a column: d_n out r for d_w_next, and
// scale D y r(y) (channel gate: its factor and slope come with the finish, as they are the same for all
// rows) or ez y r(y) for d_w_post. A thread holds those of its columns over all its rows.
template <bool F32, bool WARP, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_backward_kernel(const NormArgs p) {
    __shared__ float scratch[2][2][32];
    extern __shared__ float columns[];  // WARP: [sums][H] of the CTA
    grid_dependency_wait();
    grid_launch_dependents();
    const Place<WARP> at;
    const bool has_y = p.y != nullptr, post = p.w_post != nullptr, next = p.d_n != nullptr;
    const bool channel = p.kind == EP_GATE_CHANNEL, element = p.kind == EP_GATE_ELEMENT;
    float acc_next[NV][8], acc_y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_next[i][j] = acc_y[i][j] = 0.0f;
    int turn = 0;
    for (int t = at.row; t < p.T; t += at.step) {
        const size_t row = (size_t)t * p.vecs;
        Stream8<F32> x[NV], d[NV];
        uint4 y[NV], dn[NV], g[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            x[i].clear(), d[i].clear();
            y[i] = dn[i] = g[i] = make_uint4(0, 0, 0, 0);
            if (v >= p.vecs) continue;
            x[i].load(p.x, row + v);
            if (p.d_out) d[i].load(p.d_out, row + v);
            if (has_y) y[i] = p.y[row + v];
            if (next) dn[i] = p.d_n[row + v];
            if (channel) g[i] = static_cast<const uint4 *>(p.gate)[v];
            if (element) g[i] = static_cast<const uint4 *>(p.gate)[row + v];
        }
        const float r_y = post ? p.rstd_post[t] : 1.0f, r = next ? p.rstd_next[t] : 0.0f;
        float token_slope = 0.0f;
        const float token = p.kind == EP_GATE_TOKEN ? gate_act(static_cast<const float *>(p.gate)[t], p.sigmoid, token_slope) : 1.0f;
        float s = 0.0f, D[NV][8];  // D: first out r(out), which is near 1 at any size of the values, as r^3 is not
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            x[i].get(D[i]);
            if (!next || v >= p.vecs) continue;
            float w[8], n[8];
            if (has_y) {
                float z[8], a[8];
                unpack8(y[i], z);
                if (post) unpack8(p.w_post[v], w);
                unpack8(g[i], a);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (post) z[j] = (p.offset + w[j]) * (z[j] * r_y);
                    const float f = channel || element ? gate_act(a[j], p.sigmoid) : token;
                    D[i][j] = fmaf(p.scale * f, z[j], D[i][j]);
                }
            }
            unpack8(p.w_next[v], w);
            unpack8(dn[i], n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                D[i][j] *= r;
                s = fmaf((p.offset + w[j]) * n[j], D[i][j], s);
                acc_next[i][j] = fmaf(n[j], D[i][j], acc_next[i][j]);
            }
        }
        if (next) group_sum<WARP>(s, scratch[turn]), turn ^= 1;
        const float c = s * p.inv_h;
        float s_y = 0.0f, s_gate = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            if (v >= p.vecs) continue;
            float o[8], w[8];
            d[i].get(o);
            if (next) {
                float n[8];
                unpack8(p.w_next[v], w);
                unpack8(dn[i], n);
#pragma unroll
                for (int j = 0; j < 8; ++j) D[i][j] = fmaf(r, fmaf(p.offset + w[j], n[j], -c * D[i][j]), o[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) D[i][j] = o[j];
            }
            Stream8<F32>::store(p.d_x, row + v, D[i]);
            if (!has_y) continue;
            float yy[8], a[8], dg[8];
            unpack8(y[i], yy);
            if (post) unpack8(p.w_post[v], w);
            unpack8(g[i], a);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float wj = post ? p.offset + w[j] : 1.0f, yr = yy[j] * r_y;
                float f = token, slope = token_slope;
                if (channel || element) f = gate_act(a[j], p.sigmoid, slope);
                const float sd = p.scale * D[i][j], e = f * sd;
                acc_y[i][j] = fmaf(channel ? sd : e, yr, acc_y[i][j]);
                dg[j] = sd * (wj * yr) * slope;
                s_gate += dg[j];
                D[i][j] = wj * e;  // ew; ez where there is no norm
                s_y = fmaf(D[i][j], yr, s_y);
            }
            if (element && p.d_gate) st_v4(static_cast<uint4 *>(p.d_gate) + row + v, pack8(dg));
        }
        if (!has_y) continue;
        const bool token_sum = p.kind == EP_GATE_TOKEN && p.d_gate;
        if (post || token_sum) group_sum<WARP>(s_y, s_gate, scratch[turn]), turn ^= 1;
        if (token_sum && at.first == 0) static_cast<float *>(p.d_gate)[t] = s_gate;
        const float c_y = s_y * p.inv_h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            if (v >= p.vecs) continue;
            if (post) {
                float yy[8];
                unpack8(y[i], yy);
#pragma unroll
                for (int j = 0; j < 8; ++j) D[i][j] = r_y * fmaf(-c_y, yy[j] * r_y, D[i][j]);
            }
            st_v4(p.d_y + row + v, pack8(D[i]));
        }
    }
    // the CTA's row of partial sums
    const size_t H = (size_t)p.vecs * 8;
    const int sums = (p.next_at >= 0) + (p.y_at >= 0);
    if (sums == 0) return;
    float *out = WARP ? columns : p.partial + (size_t)blockIdx.x * sums * H;
    for (int w = 0; w < (WARP ? kNormWarps : 1); ++w) {  // warp after warp, in order
        if (WARP) __syncthreads();
        if (WARP && (int)threadIdx.x / 32 != w) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            if (v >= p.vecs) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int place = k ? p.y_at : p.next_at;
                if (place < 0) continue;
                float4 *to = reinterpret_cast<float4 *>(out + (size_t)place * H + (size_t)v * 8);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float *a = k ? &acc_y[i][4 * h] : &acc_next[i][4 * h];
                    float4 q = make_float4(a[0], a[1], a[2], a[3]);
                    if (w > 0) q.x += to[h].x, q.y += to[h].y, q.z += to[h].z, q.w += to[h].w;
                    to[h] = q;
                }
            }
        }
    }
    if constexpr (WARP) {
        __syncthreads();
        float *to = p.partial + (size_t)blockIdx.x * sums * H;
        for (int i = threadIdx.x; i < sums * (int)H; i += blockDim.x) to[i] = columns[i];
    }
}

struct FinishArgs {
    const float *partial;
    int32_t partials, H, next_at, y_at;
    const uint16_t *w_post, *gate;       // gate: of channels, else null
    float *d_w_next, *d_w_post, *d_gate;
    float offset;
    int32_t sigmoid;
};

constexpr int kFinishRows = 32;  // a CTA takes 32 columns, each warp every 32nd partial row

__global__ void __launch_bounds__(32 * kFinishRows) block_norm_finish_kernel(const FinishArgs p) {
    __shared__ float part[2][kFinishRows][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, h = blockIdx.x * 32 + lane;
    const int sums = (p.next_at >= 0) + (p.y_at >= 0);
    float a = 0.0f, b = 0.0f;
    if (h < p.H)
        for (int i = w; i < p.partials; i += kFinishRows) {
            const float *row = p.partial + (size_t)i * sums * p.H + h;
            if (p.next_at >= 0) a += row[(size_t)p.next_at * p.H];
            if (p.y_at >= 0) b += row[(size_t)p.y_at * p.H];
        }
    part[0][w][lane] = a, part[1][w][lane] = b;
    __syncthreads();
    if (w >= 2) return;  // warp 0: d_w_next, warp 1: the others
    float s = 0.0f;
    for (int i = 0; i < kFinishRows; ++i) s += part[w][i][lane];
    if (h >= p.H) return;
    if (w == 0) {
        if (p.next_at >= 0) p.d_w_next[h] = s;
        return;
    }
    if (p.y_at < 0) return;
    float slope = 1.0f, f = 1.0f, wj = 1.0f;
    if (p.gate) f = gate_act(__uint_as_float((uint32_t)p.gate[h] << 16), p.sigmoid, slope);
    if (p.w_post) wj = p.offset + __uint_as_float((uint32_t)p.w_post[h] << 16);
    if (p.d_w_post) p.d_w_post[h] = f * s;
    if (p.gate && p.d_gate) p.d_gate[h] = s * (wj * slope);
}

template <bool F32, bool WARP, int NV>
cudaError_t run_forward(const NormArgs &p, cudaStream_t s) {
    const int threads = WARP ? 32 * kNormWarps : (p.vecs + 32 * NV - 1) / (32 * NV) * 32;
    const int grid = WARP ? (p.T + kNormWarps - 1) / kNormWarps : p.T;
    return launch_dependent(block_norm_kernel<F32, WARP, NV>, dim3((unsigned)grid), dim3(threads), 0, s, p);
}
template <bool F32>
cudaError_t forward(const NormArgs &p, cudaStream_t s) {
    if (p.vecs <= 32) return run_forward<F32, true, 1>(p, s);
    if (p.vecs <= 64) return run_forward<F32, true, 2>(p, s);
    if (p.vecs <= 128) return run_forward<F32, true, 4>(p, s);
    if (p.vecs <= 1024) return run_forward<F32, false, 1>(p, s);
    return run_forward<F32, false, 2>(p, s);
}

// *partials: the CTAs, each of which leaves a row of partial sums.
template <bool F32, bool WARP, int NV, int THREADS>
cudaError_t run_backward(const NormArgs &p, int *partials, cudaStream_t s) {
    const auto kernel = block_norm_backward_kernel<F32, WARP, NV, THREADS>;
    const int threads = WARP ? THREADS : (p.vecs + 32 * NV - 1) / (32 * NV) * 32;
    const size_t smem = WARP ? (size_t)2 * p.vecs * 8 * sizeof(float) : 0;
    const int per_sm = max_blocks_per_sm((const void *)kernel, threads, smem), sms = current_device_sm_count();
    if (per_sm <= 0 || sms <= 0) return cudaErrorInvalidConfiguration;
    const int rows = WARP ? (p.T + kNormWarps - 1) / kNormWarps : p.T;
    *partials = min(min(rows, per_sm * sms), kNormMaxPartials);
    return launch_dependent(kernel, dim3((unsigned)*partials), dim3(threads), smem, s, p);
}
template <bool F32>
cudaError_t backward(const NormArgs &p, int *partials, cudaStream_t s) {
    if (p.vecs <= 32) return run_backward<F32, true, 1, 32 * kNormWarps>(p, partials, s);
    if (p.vecs <= 64) return run_backward<F32, true, 2, 32 * kNormWarps>(p, partials, s);
    if (p.vecs <= 128) return run_backward<F32, true, 4, 32 * kNormWarps>(p, partials, s);
    if (p.vecs <= 512) return run_backward<F32, false, 1, 512>(p, partials, s);
    if (p.vecs <= 1024) return run_backward<F32, false, 2, 512>(p, partials, s);
    return run_backward<F32, false, 2, 1024>(p, partials, s);
}

NormArgs norm_args(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post, const void *gate,
                   const ep_bf16 *w_next) {
    NormArgs p = {};
    p.x = x;
    p.y = reinterpret_cast<const uint4 *>(y);
    p.w_post = reinterpret_cast<const uint4 *>(w_post);
    p.w_next = reinterpret_cast<const uint4 *>(w_next);
    p.gate = gate;
    p.T = c.T;
    p.vecs = c.H / 8;
    p.kind = c.gate;
    p.sigmoid = c.gate_sigmoid;
    p.eps = c.eps;
    p.scale = c.scale;
    p.offset = c.weight_offset;
    p.inv_h = 1.0f / (float)c.H;
    p.next_at = p.y_at = -1;
    return p;
}

}  // namespace

size_t block_norm_workspace_bytes(const ep_norm_config &c) {
    return (size_t)(c.T < kNormMaxPartials ? c.T : kNormMaxPartials) * 2 * (size_t)c.H * sizeof(float);
}

cudaError_t launch_block_norm(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post, const void *gate,
                              const ep_bf16 *w_next, void *out, ep_bf16 *n, float *rstd_post, float *rstd_next,
                              cudaStream_t s) {
    NormArgs p = norm_args(c, x, y, w_post, gate, w_next);
    p.out = out;
    p.n = reinterpret_cast<uint4 *>(n);
    p.rstd_post = rstd_post;
    p.rstd_next = rstd_next;
    return c.residual_f32 ? forward<true>(p, s) : forward<false>(p, s);
}

cudaError_t launch_block_norm_backward(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post,
                                       const void *gate, const ep_bf16 *w_next, const float *rstd_post,
                                       const float *rstd_next, const void *d_out, const ep_bf16 *d_n, void *d_x, ep_bf16 *d_y,
                                       float *d_w_post, void *d_gate, float *d_w_next, float *partial, cudaStream_t s) {
    NormArgs p = norm_args(c, x, y, w_post, gate, w_next);
    p.rstd_post = const_cast<float *>(rstd_post);
    p.rstd_next = const_cast<float *>(rstd_next);
    p.d_out = d_out;
    p.d_n = reinterpret_cast<const uint4 *>(d_n);
    p.d_x = d_x;
    p.d_y = reinterpret_cast<uint4 *>(d_y);
    p.d_gate = d_gate;
    p.partial = partial;
    const bool channel = c.gate == EP_GATE_CHANNEL;
    int sums = 0;
    if (d_w_next) p.next_at = sums++;
    if (d_w_post || (channel && d_gate)) p.y_at = sums++;
    int partials = 0;
    const cudaError_t e = c.residual_f32 ? backward<true>(p, &partials, s) : backward<false>(p, &partials, s);
    if (e != cudaSuccess || sums == 0) return e;
    FinishArgs f = {};
    f.partial = partial;
    f.partials = partials;
    f.H = c.H;
    f.next_at = p.next_at;
    f.y_at = p.y_at;
    f.w_post = w_post;
    f.gate = channel ? static_cast<const uint16_t *>(gate) : nullptr;
    f.d_w_next = d_w_next;
    f.d_w_post = d_w_post;
    f.d_gate = channel ? static_cast<float *>(d_gate) : nullptr;
    f.offset = c.weight_offset;
    f.sigmoid = c.gate_sigmoid;
    return launch_dependent(block_norm_finish_kernel, dim3((unsigned)((c.H + 31) / 32)), dim3(32 * kFinishRows), 0, s, f);
}

}  // namespace ep
