// gdr_kv8_tile.cu -- attention over the 8-bit paged cache for many bf16 query rows a cached head
// (gdr_kv8_attn): the launches of the kernel in gdr_kv8_tile.cuh.

#include "gdr_kv8_tile.cuh"

namespace gdr {

cudaError_t launch_kv8_tile(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, const int *table,
                            const int *kv_len, const int *cu_q, float scale, void *out, float *lse, int S,
                            int max_q, int total_q, int Hq, int Hkv, int D, int W, int page, int N, Kv8 kv,
                            void *ws, cudaStream_t s) {
    AttnArgs a{};
    a.q = q, a.q_stride = q_stride, a.kc = static_cast<const uint8_t *>(k_cache);
    a.vc = static_cast<const uint8_t *>(v_cache);
    a.ks = k_scale, a.vs = v_scale, a.table = table, a.kv_len = kv_len;
    a.cu_q = cu_q, a.scale_log2 = fabsf(scale) * 1.4426950408889634f, a.sign = scale < 0.f ? -1.f : 1.f;
    a.out = out, a.lse = lse;
    a.S = S, a.total_q = total_q, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.W = W, a.N = N;
    a.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    a.limit_ns = wait_limit_ns();
    const int64_t rows = (int64_t)max_q * a.G;
    return kv == Kv8::E4M3 ? launch_tile_kv<Kv8::E4M3>(a, D, ws, rows, s) : launch_tile_kv<Kv8::INT8>(a, D, ws, rows, s);
}

cudaError_t take_kv8_tile_error_word(unsigned *value) { return take_attn_error_word(value); }

}  // namespace gdr
