// backward.cu -- the way back through combine and router.
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kBwdThreads = 256;

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One CTA takes JPC consecutive positions j of one token: d_y[slot[t, j]] = w[t, j] d_out[t] and
// dw[t, j] = <d_out[t], y[slot[t, j]]>. d_out is read once per CTA; the rows of y once, those of
// d_y written once, 16 bytes a thread. The products are summed in fp32: in each thread over its
// columns, then over the lanes and the warps in a fixed order.
// HBM bounds it: 4096 tokens of 7168, top-8, 1.0 GB in 150 us, 95% of the measured copy rate with the
// router's gradient behind it.
template <int JPC>
__global__ void __launch_bounds__(kBwdThreads) combine_backward_kernel(int T, int k, int vecs, const uint4 *d_out,
                                                                       const uint4 *y, const int32_t *slot,
                                                                       const float *w, uint4 *d_y, float *d_w) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int groups = (k + JPC - 1) / JPC;
    const int t = blockIdx.x / groups, j0 = blockIdx.x % groups * JPC;
    const int64_t pairs = (int64_t)T * k;
    const uint4 *d_row = d_out + (size_t)t * vecs;
    int s[JPC];
    float wj[JPC], dot[JPC];
#pragma unroll
    for (int j = 0; j < JPC; ++j) {
        const int64_t at = (int64_t)t * k + j0 + j;
        s[j] = j0 + j < k ? slot[at] : -1;
        if (s[j] >= pairs) s[j] = -1;
        wj[j] = s[j] >= 0 ? w[at] : 0.0f;
        dot[j] = 0.0f;
    }
    for (int v = threadIdx.x; v < vecs; v += blockDim.x) {
        const uint4 d = d_row[v];
        uint4 q[JPC];
#pragma unroll
        for (int j = 0; j < JPC; ++j)
            q[j] = s[j] >= 0 ? ld_stream_v4(y + (size_t)s[j] * vecs + v) : make_uint4(0, 0, 0, 0);
        const uint32_t dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < JPC; ++j) {
            if (s[j] < 0) continue;
            const uint32_t qq[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dot[j] = fmaf(bf_lo(dd[i]), bf_lo(qq[i]), dot[j]);
                dot[j] = fmaf(bf_hi(dd[i]), bf_hi(qq[i]), dot[j]);
                o[i] = bf_pair(wj[j] * bf_lo(dd[i]), wj[j] * bf_hi(dd[i]));
            }
            st_v4(d_y + (size_t)s[j] * vecs + v, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
    __shared__ float part[kBwdThreads / 32][JPC];
#pragma unroll
    for (int j = 0; j < JPC; ++j) {
        for (int d = 16; d > 0; d /= 2) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < JPC && j0 + threadIdx.x < k) {
        float sum = 0.0f;
        for (int i = 0; i < blockDim.x / 32; ++i) sum += part[i][threadIdx.x];
        d_w[(int64_t)t * k + j0 + threadIdx.x] = sum;
    }
}

constexpr int kRouteBwdWarps = 8;

// One warp per token. The gradients of the chosen experts' weights are laid out over the E experts
// in shared memory, so that the row goes out in whole lines:
//   renormalised: d_l[e] = w_e (dw_e - sum_i w_i dw_i) for the chosen experts, 0 for the others
//   otherwise:    d_l[e] = p_e (dw_e - sum_i w_i dw_i), p the softmax over all E, dw_e 0 if not chosen
// VPL: logits a lane holds. A small call is a chain of latencies, so everything is fetched at once.
template <int VPL, bool RENORM>
__global__ void __launch_bounds__(kRouteBwdWarps * 32) route_backward_kernel(int T, int E, int k, const float *logits,
                                                                            const int32_t *idx, const float *w,
                                                                            const float *d_w, float *d_logits) {
    extern __shared__ float rows[];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, t = blockIdx.x * kRouteBwdWarps + threadIdx.x / 32;
    if (t >= T) return;
    float *row = rows + threadIdx.x / 32 * E;
    const int64_t at = (int64_t)t * k + lane;
    const int e = lane < k ? idx[at] : -1;
    const float wj = lane < k ? w[at] : 0.0f, dw = lane < k ? d_w[at] : 0.0f;
    float p[VPL], top = -INFINITY, sum = 0.0f;
    if constexpr (!RENORM) {
        const float *l = logits + (size_t)t * E;
#pragma unroll
        for (int i = 0; i < VPL; ++i) p[i] = i * 32 + lane < E ? l[i * 32 + lane] : -INFINITY;
    }
    for (int i = lane; i < E; i += 32) row[i] = 0.0f;
    float inner = wj * dw;
    for (int d = 16; d > 0; d /= 2) inner += __shfl_xor_sync(0xFFFFFFFFu, inner, d);
    __syncwarp();
    if (e >= 0 && e < E) row[e] = RENORM ? wj * (dw - inner) : dw;
    __syncwarp();
    float *out = d_logits + (size_t)t * E;
    if constexpr (RENORM) {
        for (int i = lane; i < E; i += 32) out[i] = row[i];
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) top = fmaxf(top, p[i]);
        for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            p[i] = i * 32 + lane < E ? expf(p[i] - top) : 0.0f;
            sum += p[i];
        }
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i * 32 + lane < E) out[i * 32 + lane] = p[i] / sum * (row[i * 32 + lane] - inner);
    }
}

template <int VPL, bool RENORM>
cudaError_t launch_rb(const ep_config &c, const float *logits, const int32_t *idx, const float *w, const float *d_w,
                      float *d_logits, cudaStream_t s) {
    return launch_dependent(route_backward_kernel<VPL, RENORM>, dim3((unsigned)((c.T + kRouteBwdWarps - 1) / kRouteBwdWarps)),
                            dim3(kRouteBwdWarps * 32), (size_t)kRouteBwdWarps * c.E * sizeof(float), s, c.T, c.E, c.k, logits,
                            idx, w, d_w, d_logits);
}

template <int JPC>
cudaError_t launch_cb(const ep_config &c, const ep_bf16 *d_out, const ep_bf16 *y, const int32_t *slot, const float *w,
                      ep_bf16 *d_y, float *d_w, cudaStream_t s) {
    const int vecs = c.H / 8;
    const int threads = vecs >= kBwdThreads ? kBwdThreads : (vecs + 31) / 32 * 32;
    return launch_dependent(combine_backward_kernel<JPC>, dim3((unsigned)(c.T * ((c.k + JPC - 1) / JPC))), dim3(threads), 0,
                            s, c.T, c.k, vecs, reinterpret_cast<const uint4 *>(d_out), reinterpret_cast<const uint4 *>(y),
                            slot, w, reinterpret_cast<uint4 *>(d_y), d_w);
}

}  // namespace

cudaError_t launch_combine_backward(const ep_config &c, const ep_bf16 *d_out, const ep_bf16 *y, const int32_t *slot,
                                    const float *w, ep_bf16 *d_y, float *d_w, cudaStream_t s) {
    // as many positions a CTA as leave two CTAs for every SM: d_out is read once for each CTA
    const int64_t want = 2 * (int64_t)current_device_sm_count();
    const auto ctas = [&](int j) { return (int64_t)c.T * ((c.k + j - 1) / j); };
    if (ctas(8) >= want) return launch_cb<8>(c, d_out, y, slot, w, d_y, d_w, s);
    if (ctas(4) >= want) return launch_cb<4>(c, d_out, y, slot, w, d_y, d_w, s);
    if (ctas(2) >= want) return launch_cb<2>(c, d_out, y, slot, w, d_y, d_w, s);
    return launch_cb<1>(c, d_out, y, slot, w, d_y, d_w, s);
}

cudaError_t launch_route_backward(const ep_config &c, const float *logits, const int32_t *idx, const float *w,
                                  const float *d_w, float *d_logits, cudaStream_t s) {
    if (c.renormalize) return launch_rb<1, true>(c, logits, idx, w, d_w, d_logits, s);
    if (c.E <= 128) return launch_rb<4, false>(c, logits, idx, w, d_w, d_logits, s);
    if (c.E <= 256) return launch_rb<8, false>(c, logits, idx, w, d_w, d_logits, s);
    return launch_rb<kMaxE / 32, false>(c, logits, idx, w, d_w, d_logits, s);
}

}  // namespace ep
