// norm_forward.cu -- the norms around a block, forward (the kernels' frame: norm_rows.cuh).
//
// 16384 rows of 4096 with a plain residual take 85 us, 79 at the copy rate. With a norm of the block's result and a gate a row
// has two sums over the CTA instead of one, and twice the instructions: 4096 of 7168 44 us, 35 at the copy rate (issue slots
// 57 % busy, the rest waits for copies and barriers). One row of 7168: 2.4 us, a launch.
#include "norm_rows.cuh"

namespace ep {

namespace {

// AHEAD: a row's two sums over the CTA, y's and out's, are not one behind the other, but the next row's first is made with
// this row's second. That is one barrier a row, and y is asked for a row further ahead.
template <bool F32, int FORM, bool WARP, int NV, int THREADS, bool AHEAD>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : THREADS == 256 ? 3 : 1) block_norm_kernel(const NormArgs p, int stages) {
    constexpr bool kY = FORM & kFormY, kPost = FORM & kFormPost, kGate = FORM & kFormGate, kKept = kept_factors(THREADS);
    __shared__ Scratch scratch;
    extern __shared__ uint4 ring_smem[];
    clear_scratch<WARP>(scratch);
    grid_dependency_wait();
    grid_launch_dependents();
    const Place<WARP> at;
    const bool next = p.n != nullptr, element = kGate && p.kind == EP_GATE_ELEMENT, token = kY && !kGate && p.kind == EP_GATE_TOKEN;
    const bool factors = kPost || (kGate && !element);
    const Ring<F32, NV> ring(ring_smem, stages, kY, element, false, false, AHEAD);
    const auto ask_y = [&](int64_t t, uint32_t place) {
        if (t >= p.T) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * at.stride + at.first < p.vecs) ring.copy(place, 0, i, p.y, (size_t)t * p.vecs + at.first + i * at.stride);
    };
    const auto ask = [&](int64_t t, uint32_t stage) {
        if (t < p.T) {
            const size_t row = (size_t)t * p.vecs + at.first;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * at.stride + at.first >= p.vecs) continue;
                ring.copy_stream(stage, 0, i, p.x, row + i * at.stride);
                if constexpr (kY && !AHEAD) ring.copy(stage, ring.y(), i, p.y, row + i * at.stride);
                if (kGate && element) ring.copy(stage, ring.gate, i, p.gate, row + i * at.stride);
            }
        }
        copies_commit();
    };
    const auto y_squares = [&](uint32_t place) {
        uint64_t squares = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i * at.stride + at.first >= p.vecs) continue;
            const V8 v = unpack8(ring.get(place, 0, i));
            dot(squares, v, v);
        }
        return total(squares);
    };
    const auto root = [&](float sum) { return rsqrtf(fmaf(sum, p.inv_h, p.eps)); };
    if constexpr (AHEAD) ask_y(at.row, ring.y_place(0));
    for (int s = 0; s < stages; ++s) {
        if constexpr (AHEAD) ask_y((int64_t)at.row + (int64_t)(s + 1) * at.step, ring.y_place(s + 1));
        ask((int64_t)at.row + (int64_t)s * at.step, ring.stage(s));
    }
    if (kKept && factors) ring.template keep_factors<kPost, kGate>(p, at.first, at.stride);
    int s = 0, turn = 0, place = 0;  // this row's places: of the stage, and (AHEAD) of y
    float r_y = 1.0f;
    if constexpr (AHEAD) {
        copies_wait(stages - 1);
        if (at.row < p.T) r_y = root(group_sum<WARP>(y_squares(ring.y_place(0)), scratch, turn));
    }
    float token_gate = token && at.row < p.T ? static_cast<const float *>(p.gate)[at.row] : 1.0f, slope;
    for (int64_t t = at.row; t < p.T; t += at.step) {
        const size_t row = (size_t)t * p.vecs + at.first;
        const uint32_t stage = ring.stage(s);
        const float scale = token ? p.scale * gate_act(token_gate, p.sigmoid, slope) : p.scale;
        if (token && t + at.step < p.T) token_gate = static_cast<const float *>(p.gate)[t + at.step];
        copies_wait(stages - 1);
        const uint32_t y = AHEAD ? ring.y_place(place) : stage + ring.y();
        if constexpr (kPost && !AHEAD) r_y = root(group_sum<WARP>(y_squares(y), scratch, turn));
        if (kPost && p.rstd_post && at.first == 0) p.rstd_post[t] = r_y;
        V8 out[NV];
        uint64_t squares = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            if (v >= p.vecs) continue;
            out[i] = ring.get_stream(stage, 0, i);
            if constexpr (kY) {
                V8 z = unpack8(ring.get(y, 0, i));
                if constexpr (kPost) times(z, r_y);
                if (factors) times(z, ring.template get_factors<kKept, kPost, kGate>(p, i, v));
                if (kGate && element) {
                    V8 a = unpack8(ring.get(stage, ring.gate, i));
                    gate_act(a, p.sigmoid);
                    times(z, a);
                }
                add_scaled(out[i], scale, z);
                Stream8<F32>::store(p.out, row + i * at.stride, out[i]);
            }
            dot(squares, out[i], out[i]);
        }
        if constexpr (AHEAD) ask_y(t + (int64_t)(stages + 1) * at.step, y);
        ask(t + (int64_t)stages * at.step, stage);
        s = s + 1 == stages ? 0 : s + 1;
        float r;
        if constexpr (AHEAD) {
            place = place == stages ? 0 : place + 1;
            // the row after the last one: what lies there is not used
            float both[2] = {total(squares), y_squares(ring.y_place(place))};
            group_sum<WARP, 2>(both, scratch, turn);
            r = root(both[0]);
            r_y = root(both[1]);
            if (!next) continue;
        } else {
            if (!next) continue;
            r = root(group_sum<WARP>(total(squares), scratch, turn));
        }
        if (p.rstd_next && at.first == 0) p.rstd_next[t] = r;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * at.stride + at.first;
            if (v >= p.vecs) continue;
            times(out[i], r);
            weigh(out[i], __ldg(p.w_next + v), p.offset);  // weights come from L1: in registers they push others out
            st_v4(p.n + row + i * at.stride, pack8(out[i]));
        }
    }
}

// Few rows: a CTA takes one, a thread one or two vectors of it, everything asked for at once.
template <bool F32, int NV>
__global__ void __launch_bounds__(1024) block_norm_few_kernel(const NormArgs p) {
    __shared__ Scratch scratch;
    clear_scratch<false>(scratch);
    grid_dependency_wait();
    grid_launch_dependents();
    int turn = 0;
    const Place<false> at;
    const int t = at.row;
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
        uint64_t squares = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const V8 v = unpack8(y[i]);
            dot(squares, v, v);
        }
        r_y = rsqrtf(fmaf(group_sum<false>(total(squares), scratch, turn), p.inv_h, p.eps));
        if (p.rstd_post && at.first == 0) p.rstd_post[t] = r_y;
    }
    V8 out[NV];
    uint64_t squares = 0;
    float slope;
    const float scale = p.kind == EP_GATE_TOKEN ? p.scale * gate_act(token_gate, p.sigmoid, slope) : p.scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * at.stride + at.first;
        if (v >= p.vecs) continue;
        out[i] = x[i].get();
        if (has_y) {
            V8 z = unpack8(y[i]);
            if (post) {
                times(z, r_y);
                weigh(z, wp[i], p.offset);
            }
            if (p.kind == EP_GATE_CHANNEL || p.kind == EP_GATE_ELEMENT) {
                V8 a = unpack8(g[i]);
                gate_act(a, p.sigmoid);
                times(z, a);
            }
            add_scaled(out[i], scale, z);
            Stream8<F32>::store(p.out, row + v, out[i]);
        }
        dot(squares, out[i], out[i]);
    }
    if (!next) return;
    const float r = rsqrtf(fmaf(group_sum<false>(total(squares), scratch, turn), p.inv_h, p.eps));
    if (p.rstd_next && at.first == 0) p.rstd_next[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = i * at.stride + at.first;
        if (v >= p.vecs) continue;
        times(out[i], r);
        weigh(out[i], wn[i], p.offset);
        st_v4(p.n + row + v, pack8(out[i]));
    }
}

struct Forward {
    static constexpr bool kAhead = true;
    template <bool F32>
    static constexpr bool one_row() {
        return false;
    }
    template <bool F32, int FORM, bool WARP, int NV, int THREADS, bool AHEAD>
    static auto kernel() {
        return block_norm_kernel<F32, FORM, WARP, NV, THREADS, AHEAD>;
    }
};

template <bool F32, int NV>
cudaError_t few(const NormArgs &p, bool *took, cudaStream_t s) {
    const int threads = (p.vecs + 32 * NV - 1) / (32 * NV) * 32, sms = current_device_sm_count();
    // more of them than an SM's threads could hold are not asked for
    *took = p.T <= sms || (p.T <= (int64_t)sms * (2048 / threads) &&
                           p.T <= (int64_t)sms * max_blocks_per_sm((const void *)block_norm_few_kernel<F32, NV>, threads, 0));
    if (!*took) return cudaSuccess;
    return launch_dependent(block_norm_few_kernel<F32, NV>, dim3((unsigned)p.T), dim3((unsigned)threads), 0, s, p);
}
template <bool F32>
cudaError_t forward(const NormArgs &p, cudaStream_t s) {
    // a CTA for every row, as long as all of them run at once (4096 floats, normed and gated: 160 rows 4.3 us and 5.0 by the
    // other kernel, 304 5.1 and 6.6, 448, which do not, 7.8 and 7.1)
    int ctas;
    if (p.vecs > 32) {
        bool took;
        const cudaError_t e = p.vecs <= 1024 ? few<F32, 1>(p, &took, s) : few<F32, 2>(p, &took, s);
        if (took) return e;
    }
    return run_any<Forward, F32>(p, false, false, false, INT32_MAX, &ctas, s);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &p, bool f32, cudaStream_t s) { return f32 ? forward<true>(p, s) : forward<false>(p, s); }

}  // namespace ep
