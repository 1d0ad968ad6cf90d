// gdr_kv8_append.cu -- new keys and values quantised into the 8-bit paged cache
// (gdr_kv8_append).
//
// Tokens of one page follow each other in a call (slots s, s + 1, ..): such a run is the
// unit of work, for each head and for keys and values apart.  With `off` tokens in the page
// before it, the page's scale becomes s = s_req (off = 0: whatever the page held before is
// gone) or max(s_old, s_req), s_req the least power of two that holds the run's largest
// finite magnitude; the off codes already there are re-encoded if the scale grew.
//
// One warp takes a run; a token of D values is D / V lanes of 16 bytes, so a warp's loads
// and stores are whole rows.

#include "gdr_kv8.cuh"

namespace gdr {
namespace {

struct AppendArgs {
    const void *x[2];        // k, v
    uint8_t *cache[2];
    float *scale[2];
    int64_t stride[2];       // elements between tokens
    const int *slots;
    int T, H, page, N;
};

constexpr int AW = 4;   // warps a CTA

template <typename E>
__device__ __forceinline__ void load16(const E *p, float (&f)[16 / sizeof(E)]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(E) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename E, Kv8 KV, int D>
__global__ void __launch_bounds__(32 * AW) kv8_append_kernel(const AppendArgs a) {
    constexpr int V = 16 / (int)sizeof(E);      // values a lane holds of one token
    constexpr int LPT = D / V, TPW = 32 / LPT;  // lanes a token, tokens a warp step
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * AW + warp, h = blockIdx.y, w = blockIdx.z;
    if (t0 >= a.T) return;
    const int slot = a.slots[t0], P = a.page;
    if (slot < 0 || slot >= a.N * P) return;
    const int pg = slot / P, off = slot - pg * P;
    if (off > 0 && t0 > 0 && a.slots[t0 - 1] == slot - 1) return;   // inside another warp's run
    int n = 1;
    for (int i = 1; i + off < P && t0 + i < a.T; i += 32) {          // the run's length
        const int j = i + lane;
        const bool in = j + off < P && t0 + j < a.T && a.slots[t0 + j] == slot + j;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        n = i + (m == 0xffffffffu ? 32 : __ffs(~m) - 1);
        if (m != 0xffffffffu) break;
    }
    const E *x = static_cast<const E *>(a.x[w]) + (int64_t)t0 * a.stride[w] + (int64_t)h * D;
    uint8_t *blk = a.cache[w] + ((int64_t)pg * a.H + h) * P * D;
    float *sp = a.scale[w] + (int64_t)pg * a.H + h;
    const int sub = lane / LPT, d = (lane % LPT) * V;

    float amax = 0.f;
    for (int i = sub; i < n; i += TPW) {
        float f[V];
        load16<E>(x + (int64_t)i * a.stride[w] + d, f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float m = fabsf(f[k]);
            if (m <= 3.402823466e38f) amax = fmaxf(amax, m);   // infinities and NaN do not count
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float s = scale_for<KV>(amax);
    if (off > 0) {
        const float old = *sp;
        if (s > old || !(old == old)) {
            for (int i = lane * 4; i < off * D; i += 128) {
                uint32_t *c = reinterpret_cast<uint32_t *>(blk + i);
                const float2 lo = decode2<KV>(*c & 0xffffu), hi = decode2<KV>(*c >> 16);
                *c = encode2<KV>(lo.x * old / s, lo.y * old / s) | (encode2<KV>(hi.x * old / s, hi.y * old / s) << 16);
            }
        } else {
            s = old;
        }
    }
    __syncwarp();
    if (lane == 0) *sp = s;
    for (int i = sub; i < n; i += TPW) {
        float f[V];
        load16<E>(x + (int64_t)i * a.stride[w] + d, f);
        uint32_t c[V / 4];
#pragma unroll
        for (int k = 0; k < V / 4; ++k)
            c[k] = encode2<KV>(f[4 * k] / s, f[4 * k + 1] / s) | (encode2<KV>(f[4 * k + 2] / s, f[4 * k + 3] / s) << 16);
        uint32_t *o = reinterpret_cast<uint32_t *>(blk + (int64_t)(off + i) * D + d);
#pragma unroll
        for (int k = 0; k < V / 4; ++k) o[k] = c[k];
    }
}

template <typename E, Kv8 KV>
cudaError_t launch_d(const AppendArgs &a, int D, cudaStream_t s) {
    const dim3 grid((unsigned)((a.T + AW - 1) / AW), (unsigned)a.H, 2);
    if (D == 64)
        kv8_append_kernel<E, KV, 64><<<grid, 32 * AW, 0, s>>>(a);
    else
        kv8_append_kernel<E, KV, 128><<<grid, 32 * AW, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                              const int *slots, void *k_cache, void *v_cache, float *k_scale,
                              float *v_scale, int T, int H, int D, int page, int N, Elem e, Kv8 kv,
                              cudaStream_t s) {
    AppendArgs a{{k, v}, {static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache)},
                 {k_scale, v_scale}, {k_stride, v_stride}, slots, T, H, page, N};
    if (e == Elem::BF16)
        return kv == Kv8::E4M3 ? launch_d<__nv_bfloat16, Kv8::E4M3>(a, D, s)
                               : launch_d<__nv_bfloat16, Kv8::INT8>(a, D, s);
    return kv == Kv8::E4M3 ? launch_d<float, Kv8::E4M3>(a, D, s) : launch_d<float, Kv8::INT8>(a, D, s);
}

}  // namespace gdr
