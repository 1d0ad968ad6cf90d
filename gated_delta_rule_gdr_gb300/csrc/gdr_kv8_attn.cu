// gdr_kv8_attn.cu -- attention over the 8-bit paged cache (gdr_kv8_attn).
//
// Query i of request s (n queries, the last n of kv tokens) sees keys j <= kv - n + i:
//   x_j = scale ks_page(j) (q . kcode_j),  o = sum_j softmax(x)_j vs_page(j) vcode_j,
//   lse = ln sum_j e^x_j;  a query that sees nothing gives o = 0 and lse = -inf.
//
// One warp takes one (query, head): a lane per key of a block of 32, a running maximum and
// sum, the values taken lane = dimension with each key's weight broadcast.

#include "gdr_kv8.cuh"

#include <cmath>

namespace gdr {
namespace {

struct AttnArgs {
    const void *q;
    int64_t q_stride;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int *table, *kv_len, *cu_q;
    float scale;
    void *out;
    float *lse;
    int S, total_q, Hq, Hkv, W, page, N;
};

template <typename E> __device__ __forceinline__ float to_f(E x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename E, Kv8 KV, int D>
__global__ void __launch_bounds__(128) kv8_rows_kernel(const AttnArgs a) {
    __shared__ float s_q[4][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 4 + warp;
    if (row >= (int64_t)a.total_q * a.Hq) return;
    const int t = (int)(row / a.Hq), hq = (int)(row % a.Hq), h = hq / (a.Hq / a.Hkv);
    int s = t, i = 0, n = 1;
    if (a.cu_q) {
        int lo = 0, hi = a.S;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_q[mid] <= t) lo = mid; else hi = mid;
        }
        s = lo;
        i = t - a.cu_q[s];
        n = a.cu_q[s + 1] - a.cu_q[s];
        if (i < 0 || i >= n) return;   // a row outside every request
    }
    const int kv = (int)min((int64_t)max(a.kv_len[s], 0), (int64_t)a.W * a.page);
    const int end = min(kv, max(0, kv - n + i + 1));
    const E *q = static_cast<const E *>(a.q) + (int64_t)t * a.q_stride + (int64_t)hq * D;
    for (int d = lane; d < D; d += 32) s_q[warp][d] = to_f<E>(q[d]) * a.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int j0 = 0; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        const int pg = j < end ? a.table[(int64_t)s * a.W + j / a.page] : -1;
        float x = -INFINITY;
        int64_t base = 0;
        float vs = 0.f;
        if (pg >= 0 && pg < a.N) {
            base = (((int64_t)pg * a.Hkv + h) * a.page + j % a.page) * D;
            vs = a.vs[(int64_t)pg * a.Hkv + h];
            x = 0.f;
            for (int d = 0; d < D; d += 4) {
                const uint32_t c = *reinterpret_cast<const uint32_t *>(a.kc + base + d);
                const float2 u = decode2<KV>(c & 0xffffu), w = decode2<KV>(c >> 16);
                x += s_q[warp][d] * u.x + s_q[warp][d + 1] * u.y + s_q[warp][d + 2] * w.x + s_q[warp][d + 3] * w.y;
            }
            x *= a.ks[(int64_t)pg * a.Hkv + h];
        }
        const unsigned there = __ballot_sync(0xffffffffu, pg >= 0 && pg < a.N);
        float mx = x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx);
        if (there == 0) continue;
        const float ref = mn == -INFINITY ? 0.f : mn;   // every score NaN: the weights are too
        const float al = __expf(m - ref), p = __expf(x - ref);
        m = mn;
        float sum = p;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * al + sum;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] *= al;
        const float pv = p * vs;
        for (int k = 0; k < 32; ++k) {
            if (!(there >> k & 1)) continue;
            const float w = __shfl_sync(0xffffffffu, pv, k);
            const int64_t b = __shfl_sync(0xffffffffu, base, k);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) o[e] += w * decode2<KV>(a.vc[b + 32 * e + lane]).x;
        }
    }
    E *out = static_cast<E *>(a.out) + row * D;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) out[32 * e + lane] = from_f<E>(l == 0.f ? 0.f : o[e] / l);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename E, Kv8 KV>
cudaError_t launch_rows(const AttnArgs &a, int D, cudaStream_t s) {
    const int64_t rows = (int64_t)a.total_q * a.Hq;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (D == 64)
        kv8_rows_kernel<E, KV, 64><<<grid, 128, 0, s>>>(a);
    else
        kv8_rows_kernel<E, KV, 128><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t kv8_attn_workspace_bytes(int, int, int, int, int, int, Elem) { return 0; }

cudaError_t launch_kv8_attn(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, const int *table,
                            const int *kv_len, const int *cu_q, float scale, void *out, float *lse, int S,
                            int max_q, int total_q, int Hq, int Hkv, int D, int W, int page, int N, Elem e,
                            Kv8 kv, void *ws, cudaStream_t s) {
    (void)max_q;
    (void)ws;
    const AttnArgs a{q, q_stride, static_cast<const uint8_t *>(k_cache),
                     static_cast<const uint8_t *>(v_cache), k_scale, v_scale, table, kv_len, cu_q, scale,
                     out, lse, S, total_q, Hq, Hkv, W, page, N};
    if (e == Elem::BF16)
        return kv == Kv8::E4M3 ? launch_rows<__nv_bfloat16, Kv8::E4M3>(a, D, s)
                               : launch_rows<__nv_bfloat16, Kv8::INT8>(a, D, s);
    return kv == Kv8::E4M3 ? launch_rows<float, Kv8::E4M3>(a, D, s) : launch_rows<float, Kv8::INT8>(a, D, s);
}

}  // namespace gdr
