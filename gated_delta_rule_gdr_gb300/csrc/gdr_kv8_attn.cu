// gdr_kv8_attn.cu -- attention over the 8-bit paged cache (gdr_kv8_attn): the kernel for few query rows a
// cached head and for fp32 (gdr_kv8_split.cuh), or the one for many (gdr_kv8_tile.cu).

#include "gdr_kv8_split.cuh"

namespace gdr {

size_t kv8_attn_workspace_bytes(int, int max_q, int, int Hq, int Hkv, int D, Elem e) {
    return shape_workspace_bytes(shape_of(max_q, Hq / Hkv, e), D);
}

cudaError_t launch_kv8_attn(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, const int *table,
                            const int *kv_len, const int *cu_q, float scale, void *out, float *lse, int S,
                            int max_q, int total_q, int Hq, int Hkv, int D, int W, int page, int N, Elem e,
                            Kv8 kv, void *ws, cudaStream_t s) {
    const Shape sh = shape_of(max_q, Hq / Hkv, e);
    if (sh == Shape::TILE)
        return launch_kv8_tile(q, q_stride, k_cache, v_cache, k_scale, v_scale, table, kv_len, cu_q, scale, out,
                               lse, S, max_q, total_q, Hq, Hkv, D, W, page, N, kv, ws, s);
    AttnArgs a{};
    a.q = q, a.q_stride = q_stride, a.ks = k_scale, a.vs = v_scale, a.table = table, a.kv_len = kv_len;
    a.cu_q = cu_q, a.scale_log2 = fabsf(scale) * 1.4426950408889634f, a.sign = scale < 0.f ? -1.f : 1.f;
    a.out = out, a.lse = lse;
    a.S = S, a.total_q = total_q, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.W = W, a.N = N;
    a.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    a.limit_ns = wait_limit_ns();
    return launch_split_any(a, sh, k_cache, v_cache, D, e, kv, ws, (int64_t)max_q * a.G, s);
}

cudaError_t take_kv8_split_error_word(unsigned *value) { return take_attn_error_word(value); }

}  // namespace gdr
