/* Calls ep_expert_ffn over and over, without the interpreter's lock; built and called by
 * test_gpu_expert_threads.py. Returns the first status that is not 0, and the call's number. */
typedef int (*ffn_call)(const void *cfg, const void *rows, const void *offset, const void *w_gate, const void *w_up,
                        const void *w_down, void *g, void *u, void *h, void *y, void *stream);

int call_often(ffn_call f, int times, int *at, const void *cfg, const void *rows, const void *offset, const void *w,
               const void *w_down, void *h, void *y, void *stream) {
    for (int i = 0; i < times; ++i) {
        const int status = f(cfg, rows, offset, w, w, w_down, 0, 0, h, y, stream);
        if (status) {
            *at = i;
            return status;
        }
    }
    return 0;
}
