// norm_backward.cu -- the norms around a block, backward (the kernels' frame: norm_rows.cuh).
//
// 16384 rows of 4096 with a plain residual, bf16: 140 us with the joining of the CTAs' sums over rows (5), 119 at the copy
// rate; normed as well 155. 4096 of 7168: 67, normed and gated by channels 87 (52); fp32 110 and 123 (78).
#include "norm_rows.cuh"

namespace ep {

namespace {

// The sums over rows that it keeps, a value a column: d_n out r for d_w_next, and scale D y r(y) (channel
// gate: its factor and slope come with the finish, as they are the same for all rows) or ez y r(y) for d_w_post. A
// thread holds those of its columns over all its rows.
template <bool F32, int FORM, bool WARP, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 320 ? 2 : 1) block_norm_backward_kernel(const NormArgs p, int stages) {
    constexpr bool kY = FORM & kFormY, kPost = FORM & kFormPost, kGate = FORM & kFormGate, kKept = kept_factors(THREADS);
    __shared__ Scratch scratch;
    extern __shared__ uint4 ring_smem[];  // at the end, WARP: [sums][H] of the CTA
    clear_scratch<WARP>(scratch);
    grid_dependency_wait();
    grid_launch_dependents();
    const Place<WARP> at;
    const bool next = p.d_n != nullptr, has_d = p.d_out != nullptr;
    const bool channel = kGate && p.kind == EP_GATE_CHANNEL, element = kGate && !channel, token = kY && !kGate && p.kind == EP_GATE_TOKEN;
    const bool factors = kPost || (kGate && !element);
    const Ring<F32, NV> ring(ring_smem, stages, kY, element, has_d, next);
    const auto ask = [&](int64_t t, uint32_t stage) {
        if (t < p.T) {
            const size_t row = (size_t)t * p.vecs + at.first;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * at.stride + at.first >= p.vecs) continue;
                const size_t v = row + i * at.stride;
                if (next) ring.copy_stream(stage, 0, i, p.x, v);
                if constexpr (kY) ring.copy(stage, ring.y(), i, p.y, v);
                if (kGate && element) ring.copy(stage, ring.gate, i, p.gate, v);
                if (has_d) ring.copy_stream(stage, ring.d_out, i, p.d_out, v);
                if (next) ring.copy(stage, ring.d_n, i, p.d_n, v);
            }
        }
        copies_commit();
    };
    for (int s = 0; s < stages; ++s) ask((int64_t)at.row + (int64_t)s * at.step, ring.stage(s));
    if (kKept && factors) ring.template keep_factors<kPost, kGate>(p, at.first, at.stride);
    V8 acc_next[NV], acc_y[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc_next[i].p[j] = acc_y[i].p[j] = 0;
    // a row's scalars, asked for a row ahead
    float r_y = 1.0f, r = 0.0f, token_gate = 1.0f;
    const auto scalars = [&](int64_t t) {
        if (t >= p.T) return;
        if (kPost) r_y = p.rstd_post[t];
        if (next) r = p.rstd_next[t];
        if (token) token_gate = static_cast<const float *>(p.gate)[t];
    };
    scalars(at.row);
    int s = 0, turn = 0;
    for (int64_t t = at.row; t < p.T; t += at.step) {
        const size_t row = (size_t)t * p.vecs + at.first;
        const uint32_t stage = ring.stage(s);
        const float ry = r_y, rn = r;
        float token_slope = 0.0f;
        const float scale = token ? p.scale * gate_act(token_gate, p.sigmoid, token_slope) : p.scale;  // with a token's gate
        scalars(t + at.step);
        copies_wait(stages - 1);
        // A piece's place is filled for a row ahead as soon as the pieces of its array have been read for the last time, as
        // otherwise too little is in flight (floats, 8192 rows of 7168, both directions, 411 -> 365 us; bf16, 16384 of 4096,
        // normed, backward 165 -> 155, 4096 of 2048 28.3 -> 26.9).
        const int64_t t_ahead = t + (int64_t)stages * at.step;
        const bool more = t_ahead < p.T;
        const size_t ahead = (size_t)t_ahead * p.vecs + at.first;
        // D: first out r(out), which is near 1 at any size of the values, as r^3 is not; gn beside it
        V8 D[NV], gn[NV];
        float c = 0.0f;
        if (next) {
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * at.stride + at.first;
                if (v >= p.vecs) continue;
                D[i] = ring.get_stream(stage, 0, i);
                if constexpr (kY) {
                    V8 z = unpack8(ring.get(stage, ring.y(), i));
                    if constexpr (kPost) times(z, ry);
                    if (factors) times(z, ring.template get_factors<kKept, kPost, kGate>(p, i, v));
                    if (kGate && element) {
                        V8 a = unpack8(ring.get(stage, ring.gate, i));
                        gate_act(a, p.sigmoid);
                        times(z, a);
                    }
                    add_scaled(D[i], scale, z);
                }
                times(D[i], rn);
                gn[i] = unpack8(ring.get(stage, ring.d_n, i));
                add_product(acc_next[i], gn[i], D[i]);
                weigh(gn[i], __ldg(p.w_next + v), p.offset);
                dot(sum, gn[i], D[i]);
            }
            if (more)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (i * at.stride + at.first >= p.vecs) continue;
                    ring.copy_stream(stage, 0, i, p.x, ahead + i * at.stride);
                    ring.copy(stage, ring.d_n, i, p.d_n, ahead + i * at.stride);
                }
            c = group_sum<WARP>(total(sum), scratch, turn) * p.inv_h;
        }
        uint64_t sum_y = 0, sum_gate = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            if (v >= p.vecs) continue;
            V8 d;
            if (has_d) {
                d = ring.get_stream(stage, ring.d_out, i);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) d.p[j] = 0;
            }
            if (next) {
                add_scaled(gn[i], -c, D[i]);
                add_scaled(d, rn, gn[i]);
            }
            Stream8<F32>::store(p.d_x, row + i * at.stride, d);
            if constexpr (kY) {
                if (kPost || kGate || token) {
                    V8 z = unpack8(ring.get(stage, ring.y(), i));  // y r(y)
                    if constexpr (kPost) times(z, ry);
                    V8 sd = d;
                    times(sd, p.scale);
                    if (channel) {
                        add_product(acc_y[i], sd, z);
                        d = sd;
                    } else if (kGate) {
                        V8 a = unpack8(ring.get(stage, ring.gate, i)), slope;
                        gate_act(a, p.sigmoid, slope);
                        d = sd;
                        times(d, a);  // ez
                        if (p.d_gate) {
                            times(sd, z);
                            if constexpr (kPost) times(sd, ring.template get_factors<kKept, kPost, kGate>(p, i, v));
                            times(sd, slope);
                            st_v4(static_cast<uint4 *>(p.d_gate) + row + i * at.stride, pack8(sd));
                        }
                    } else {
                        times(d, scale);  // ez
                        if (token) {
                            times(sd, z);
                            if constexpr (kPost) times(sd, ring.template get_factors<kKept, kPost, kGate>(p, i, v));
#pragma unroll
                            for (int j = 0; j < 4; ++j) sum_gate = add2(sum_gate, sd.p[j]);
                        }
                    }
                    if (kPost && !channel) add_product(acc_y[i], d, z);
                    if (factors) times(d, ring.template get_factors<kKept, kPost, kGate>(p, i, v));  // ew
                    if constexpr (kPost) dot(sum_y, d, z);
                } else {
                    times(d, scale);
                }
                D[i] = d;
            }
        }
        if (more && has_d)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i * at.stride + at.first < p.vecs) ring.copy_stream(stage, ring.d_out, i, p.d_out, ahead + i * at.stride);
        if constexpr (kY) {
            float s_y = total(sum_y), s_gate = total(sum_gate);
            const bool token_sum = token && p.d_gate;
            if (token_sum) {
                float both[2] = {s_y, s_gate};
                group_sum<WARP, 2>(both, scratch, turn);
                s_y = both[0];
                if (at.first == 0) static_cast<float *>(p.d_gate)[t] = both[1] * token_slope;
            } else if (kPost) {
                s_y = group_sum<WARP>(s_y, scratch, turn);
            }
            const float c_y = s_y * p.inv_h * ry;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * at.stride + at.first >= p.vecs) continue;
                if constexpr (kPost) {
                    add_scaled(D[i], -c_y, unpack8(ring.get(stage, ring.y(), i)));
                    times(D[i], ry);
                }
                if (more) {
                    ring.copy(stage, ring.y(), i, p.y, ahead + i * at.stride);
                    if (kGate && element) ring.copy(stage, ring.gate, i, p.gate, ahead + i * at.stride);
                }
                st_v4(p.d_y + row + i * at.stride, pack8(D[i]));
            }
        }
        copies_commit();
        s = s + 1 == stages ? 0 : s + 1;
    }
    // the CTA's row of partial sums
    const size_t H = (size_t)p.vecs * 8;
    const int sums = (p.next_at >= 0) + (p.y_at >= 0);
    if (sums == 0) return;
    float *columns = reinterpret_cast<float *>(ring_smem);
    float *out = WARP ? columns : p.partial + (size_t)blockIdx.x * sums * H;
    copies_wait(0);
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
                    const V8 &a = k ? acc_y[i] : acc_next[i];
                    float4 q = make_float4(low(a.p[2 * h]), high(a.p[2 * h]), low(a.p[2 * h + 1]), high(a.p[2 * h + 1]));
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

struct Backward {
    static constexpr bool kAhead = false;
    template <bool F32>
    static constexpr bool one_row() {
        return F32;
    }
    template <bool F32, int FORM, bool WARP, int NV, int THREADS, bool AHEAD>
    static auto kernel() {
        return block_norm_backward_kernel<F32, FORM, WARP, NV, THREADS>;
    }
};

}  // namespace

cudaError_t launch_norm_backward(const NormArgs &p, bool f32, int most, int *ctas, cudaStream_t s) {
    const bool d = p.d_out != nullptr, n = p.d_n != nullptr;
    return f32 ? run_any<Backward, true>(p, d, n, true, most, ctas, s)
               : run_any<Backward, false>(p, d, n, true, most, ctas, s);
}

}  // namespace ep
