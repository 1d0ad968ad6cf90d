// gdr_kv8_shared_e4m3.cu -- attention of requests that share a prefix (gdr_kv8_attn_shared): its passes in
// the kernel for many query rows a cached head, e4m3 codes (a file for each type, to compile side by side).

#include "gdr_kv8_tile.cuh"

namespace gdr {

cudaError_t launch_kv8_shared_e4m3(const KvSharedCall &c, bool first, float *pre_o, float2 *pre_ml, void *parts, cudaStream_t s) {
    if (first) {
        SharedArgs<true> a = shared_args<true>(c, pre_o, pre_ml);
        return launch_tile_kv<Kv8::E4M3>(a, c.D, parts, (int64_t)c.max_group_q * a.G, s);
    }
    SharedArgs<false> a = shared_args<false>(c, pre_o, pre_ml);
    return launch_tile_kv<Kv8::E4M3>(a, c.D, parts, (int64_t)c.max_q * a.G, s);
}

cudaError_t take_kv8_shared_e4m3_error_word(unsigned *value) { return take_attn_error_word(value); }

}  // namespace gdr
