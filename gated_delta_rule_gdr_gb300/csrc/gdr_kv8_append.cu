// gdr_kv8_append.cu -- new keys and values quantised into the 8-bit paged cache
// (gdr_kv8_append).
//
// Tokens of one page follow each other in a call (slots s, s + 1, ..): such a run is the
// unit of work, for each head and for keys and values apart.  With `off` tokens in the page
// before it, the page's scale becomes s = s_req (off = 0: whatever the page held before is
// gone) or max(s_old, s_req), s_req the least power of two that holds the run's largest
// finite magnitude; the off codes already there are re-encoded if the scale grew.
//
// Bound: bytes.  Measured: 16384 tokens x 8 heads x 128 bf16 values (101 MB, 14.8 us at the copy
// rate) 20.2 us = 5.0 TB/s; 37 requests of up to 400 fp32 tokens (24 MB, 3.6 us) 6.9 us; 64
// single tokens 2.7 us, a launch.  A run's values are
// read once, held in registers as they came (16 bytes a piece) through the maximum, then
// scaled, rounded and stored.  The maximum is taken on the bit patterns without their signs,
// two bf16 values an operation; it also tells when a value is not finite, which alone costs a
// second look.  Runs of at most 256 pieces are a warp's (one token, short chunks: as many
// runs in flight as there are warps), longer ones the whole CTA's.  A CTA looks for the runs
// that begin in its window of tokens; the window is short where there are few tokens, so that
// a decode step spreads over the device.  A lane's pieces of keys and values together are more
// than the fp32 instances' registers hold beside the division of the slow path: they spill 96 to
// 416 bytes a thread.

#include "gdr_kv8.cuh"

namespace gdr {
namespace {

struct AppendArgs {
    const void *x[2];        // k, v
    uint8_t *cache[2];
    float *scale[2];
    int64_t stride[2];       // elements between tokens
    const int *slots;
    int T, H, D, page_log2, N;
    int window, pieces_log2; // tokens a CTA looks for runs in; 16-byte pieces of a token
};

constexpr int ANT = 256;          // threads
constexpr int MAXW = 128;         // tokens of the longest window
// Pieces a lane holds of a warp's run, of keys and of values (fewer where the CTA takes the
// long ones, so that more CTAs are resident); CTAs an SM.
template <int MAXP> constexpr int WPIECES = MAXP == 1 ? 8 : MAXP <= 8 ? 4 : 8;
template <int MAXP> constexpr int RESIDENT = MAXP == 4 ? 3 : MAXP <= 8 ? 2 : 1;

// The largest magnitude of a piece as a bit pattern, folded into `m`: fp32 patterns, or the
// larger half of packed bf16 ones (kept apart until fold()).
template <typename E> __device__ __forceinline__ uint32_t piece_max(uint32_t m, uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = sizeof(E) == 4 ? max(m, w[i] & 0x7fffffffu) : __vmaxu2(m, w[i] & 0x7fff7fffu);
    return m;
}
template <typename E> __device__ __forceinline__ uint32_t fold(uint32_t m) {   // as an fp32 pattern
    return sizeof(E) == 4 ? m : max(m & 0xffff0000u, m << 16);
}
constexpr uint32_t kInfBits = 0x7f800000u;
// The same over finite values only.
template <typename E> __device__ __forceinline__ uint32_t piece_max_finite(uint32_t m, uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < (sizeof(E) == 4 ? 1 : 2); ++k) {
            const uint32_t b = (sizeof(E) == 4 ? w[i] : k ? w[i] & 0xffff0000u : w[i] << 16) & 0x7fffffffu;
            if (b < kInfBits) m = max(m, b);
        }
    return m;
}

// 1 / s where s is a power of two (scaling by it then is the division, correctly rounded), or
// 0: divide (a cache whose scales were made elsewhere).
__device__ __forceinline__ float exact_inverse(float s) {
    const uint32_t u = __float_as_uint(s);
    const bool pow2 = (u & 0x807fffffu) == 0 && u >= 0x00800000u && u < 0x7f000000u;
    return pow2 ? __uint_as_float(0x7f000000u - u) : 0.f;
}
// Codes of four finite values; for int8 within +-127 (a scale below the largest one holds them).
template <Kv8 KV> __device__ __forceinline__ uint32_t encode4_plain(float y0, float y1, float y2, float y3) {
    if constexpr (KV == Kv8::E4M3) {
        uint32_t r;
        asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t}"
            : "=r"(r)
            : "f"(y0), "f"(y1), "f"(y2), "f"(y3));
        return r;
    } else {      // adding 1.5 2^23 rounds to the nearest integer, ties to even, in the low byte
        constexpr float big = 12582912.f;
        const uint32_t a = __byte_perm(__float_as_uint(y0 + big), __float_as_uint(y1 + big), 0x0040);
        const uint32_t b = __byte_perm(__float_as_uint(y2 + big), __float_as_uint(y3 + big), 0x0040);
        return __byte_perm(a, b, 0x5410);
    }
}
// Codes of a piece (8 bf16 or 4 fp32 values).  PLAIN: the values are what encode4_plain takes and
// s is 1 / scale exactly; else s is the scale.
template <typename E, Kv8 KV, bool PLAIN>
__device__ __forceinline__ void store_piece(uint8_t *dst, uint4 u, float s) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    auto four = [&](uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) -> uint32_t {
        const float f0 = __uint_as_float(b0), f1 = __uint_as_float(b1), f2 = __uint_as_float(b2), f3 = __uint_as_float(b3);
        if constexpr (PLAIN) return encode4_plain<KV>(f0 * s, f1 * s, f2 * s, f3 * s);
        return encode2<KV>(f0 / s, f1 / s) | (encode2<KV>(f2 / s, f3 / s) << 16);
    };
    if constexpr (sizeof(E) == 4)
        *reinterpret_cast<uint32_t *>(dst) = four(w[0], w[1], w[2], w[3]);
    else
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(four(w[0] << 16, w[0] & 0xffff0000u, w[1] << 16, w[1] & 0xffff0000u),
                       four(w[2] << 16, w[2] & 0xffff0000u, w[3] << 16, w[3] & 0xffff0000u));
}
// This thread's pieces first, first + step, .. of a run (P of them at most) to the page.
template <typename E, Kv8 KV, int P>
__device__ __forceinline__ void store_run(uint8_t *dst, const uint4 (&u)[P], int first, int step, int pieces, float s,
                                          bool finite) {
    constexpr int V = 16 / (int)sizeof(E);
    const float inv = exact_inverse(s);
    if (finite && inv != 0.f) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (first + step * i < pieces) store_piece<E, KV, true>(dst + (first + step * i) * V, u[i], inv);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (first + step * i < pieces) store_piece<E, KV, false>(dst + (first + step * i) * V, u[i], s);
    }
}

// The page's scale for a run whose largest finite magnitude is amax, and whether the codes
// before the run have to be re-encoded (from `old`).
template <Kv8 KV>
__device__ __forceinline__ float page_scale(float amax, int off, float old, bool &grew) {
    const float req = scale_for<KV>(amax);
    grew = off > 0 && (req > old || !(old == old));
    return off == 0 || grew ? req : old;
}
template <Kv8 KV>
__device__ __forceinline__ void re_encode(uint8_t *blk, int bytes, float old, float s, int first, int step) {
    for (int i = first * 4; i < bytes; i += step * 4) {
        uint32_t *c = reinterpret_cast<uint32_t *>(blk + i);
        const float2 lo = decode2<KV>(*c & 0xffffu), hi = decode2<KV>(*c >> 16);
        *c = encode2<KV>(lo.x * old / s, lo.y * old / s) | (encode2<KV>(hi.x * old / s, hi.y * old / s) << 16);
    }
}

// A run's keys and values, by `step` threads of which this is `first`; all_max folds a maximum
// over them.
template <typename E, Kv8 KV, int P, typename AllMax>
__device__ __forceinline__ void append_run(const AppendArgs &a, int t, int slot, int n, int h, int first, int step,
                                           AllMax all_max) {
    const int pg = slot >> a.page_log2, off = slot & ((1 << a.page_log2) - 1), lpt = a.pieces_log2, pieces = n << lpt;
    const int64_t ph = (int64_t)pg * a.H + h, base = ((ph << a.page_log2) + off) * a.D;
    const int d0 = first & ((1 << lpt) - 1), row0 = first >> lpt, rows = step >> lpt;   // step is whole tokens
    uint4 u[2][P];
    float old[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const E *>(a.x[w]) + (int64_t)(t + row0) * a.stride[w] +
                                                           (int64_t)h * a.D) + d0;
        const int64_t next = (int64_t)rows * a.stride[w] * (int)sizeof(E) / 16;
#pragma unroll
        for (int i = 0; i < P; ++i)
            u[w][i] = first + step * i < pieces ? src[next * i] : make_uint4(0, 0, 0, 0);
        old[w] = off > 0 ? a.scale[w][ph] : 0.f;
    }
    uint32_t m[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < P; ++i) m[w] = piece_max<E>(m[w], u[w][i]);
        m[w] = fold<E>(m[w]);
    }
    all_max(m);
    const bool finite = m[0] < kInfBits && m[1] < kInfBits;
    if (!finite) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            m[w] = 0;
#pragma unroll
            for (int i = 0; i < P; ++i) m[w] = piece_max_finite<E>(m[w], u[w][i]);
        }
        all_max(m);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        bool grew;
        const float s = page_scale<KV>(__uint_as_float(m[w]), off, old[w], grew);
        if (grew) re_encode<KV>(a.cache[w] + base - off * a.D, off * a.D, old[w], s, first, step);
        if (first == 0) a.scale[w][ph] = s;
        store_run<E, KV, P>(a.cache[w] + base, u[w], first, step, pieces, s,
                            finite && (KV == Kv8::E4M3 || __uint_as_float(m[w]) <= 127.f * s));
    }
}

template <typename E, Kv8 KV, int MAXP>
__global__ void __launch_bounds__(ANT, RESIDENT<MAXP>) kv8_append_kernel(const AppendArgs a) {
    constexpr int WP = WPIECES<MAXP>;
    __shared__ int s_slot[1 + MAXW + 128];      // of the token before the window, the window, a page more
    __shared__ int s_lead[MAXW], s_long[MAXW], s_len[MAXW], s_count[2];
    __shared__ uint32_t s_red[2][ANT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int W = a.window, t0 = blockIdx.x * W, h = blockIdx.y, P = 1 << a.page_log2;
    if (tid < 2) s_count[tid] = 0;
    for (int i = tid; i < 1 + W + P; i += ANT) {
        const int t = t0 - 1 + i;
        const int slot = t >= 0 && t < a.T ? a.slots[t] : -1;
        s_slot[i] = slot < (a.N << a.page_log2) ? slot : -1;
    }
    __syncthreads();
    // a run begins at a slot that does not follow its predecessor's, or at a page's first place
    if (tid < W) {
        const int slot = s_slot[1 + tid];
        if (slot >= 0 && ((slot & (P - 1)) == 0 || s_slot[tid] != slot - 1)) s_lead[atomicAdd(&s_count[0], 1)] = tid;
    }
    __syncthreads();
    const int leads = s_count[0];
    // ---- a warp's runs
    for (int r = warp; r < leads; r += ANT / 32) {
        const int j = s_lead[r], slot = s_slot[1 + j], room = P - (slot & (P - 1));
        int n = 1;
        while (n < room) {
            const int i = n + lane;
            const unsigned m = __ballot_sync(0xffffffffu, i < room && s_slot[1 + j + i] == slot + i);
            n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            if (m != 0xffffffffu) break;
        }
        if (MAXP > 1 && (n << a.pieces_log2) > 32 * WP) {
            if (lane == 0) {
                const int at = atomicAdd(&s_count[1], 1);
                s_long[at] = j;
                s_len[at] = n;
            }
            continue;
        }
        append_run<E, KV, WP>(a, t0 + j, slot, n, h, lane, 32, [&](uint32_t (&m)[2]) {
            m[0] = __reduce_max_sync(0xffffffffu, m[0]);
            m[1] = __reduce_max_sync(0xffffffffu, m[1]);
        });
    }
    if constexpr (MAXP > 1) {        // MAXP 1: no page holds more than a warp's pieces
        __syncthreads();
        const int longs = s_count[1];
        // ---- the CTA's
#pragma unroll 1
        for (int r = 0; r < longs; ++r)
            append_run<E, KV, MAXP>(a, t0 + s_long[r], s_slot[1 + s_long[r]], s_len[r], h, tid, ANT, [&](uint32_t (&m)[2]) {
                m[0] = __reduce_max_sync(0xffffffffu, m[0]);
                m[1] = __reduce_max_sync(0xffffffffu, m[1]);
                __syncthreads();
                if (lane < 2) s_red[lane][warp] = lane ? m[1] : m[0];
                __syncthreads();
#pragma unroll
                for (int w = 0; w < ANT / 32; ++w) {
                    m[0] = max(m[0], s_red[0][w]);
                    m[1] = max(m[1], s_red[1][w]);
                }
            });
    }
}

// Pieces a thread holds of a CTA's longest run: a page's.
template <typename E, Kv8 KV>
cudaError_t launch_p(const AppendArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.T + a.window - 1) / a.window), (unsigned)a.H);
    const int need = ((1 << (a.page_log2 + a.pieces_log2)) + ANT - 1) / ANT;
    if (need <= 1)
        kv8_append_kernel<E, KV, 1><<<grid, ANT, 0, s>>>(a);
    else if (need <= 4)
        kv8_append_kernel<E, KV, 4><<<grid, ANT, 0, s>>>(a);
    else if (need <= 8)
        kv8_append_kernel<E, KV, 8><<<grid, ANT, 0, s>>>(a);
    else
        kv8_append_kernel<E, KV, 16><<<grid, ANT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                              const int *slots, void *k_cache, void *v_cache, float *k_scale,
                              float *v_scale, int T, int H, int D, int page, int N, Elem e, Kv8 kv,
                              cudaStream_t s) {
    // A window of 8 tokens gives every warp one, for up to about 4 CTAs an SM; more tokens
    // take longer windows, up to a page's run where that is the CTA's and several short pages'
    // where it is a warp's.  64 single tokens: 2.9 us at 8, 9.9 at the longest; 16384 tokens of
    // prompts: 41 and 20.5; 37 ragged fp32 requests: 22.9 and 6.5 (7.1 at what this chooses).
    int window = 8;
    const int most = page * D * (e == Elem::BF16 ? 2 : 4) > 4096 ? page : MAXW;
    while (window < most && (int64_t)T * H > (int64_t)window * 608) window *= 2;
    const int row_bytes = D * (e == Elem::BF16 ? 2 : 4);
    int lpt = 0;
    while ((16 << lpt) < row_bytes) ++lpt;
    AppendArgs a{{k, v}, {static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache)},
                 {k_scale, v_scale}, {k_stride, v_stride}, slots, T, H, D, page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7, N, window, lpt};
    if (e == Elem::BF16)
        return kv == Kv8::E4M3 ? launch_p<__nv_bfloat16, Kv8::E4M3>(a, s) : launch_p<__nv_bfloat16, Kv8::INT8>(a, s);
    return kv == Kv8::E4M3 ? launch_p<float, Kv8::E4M3>(a, s) : launch_p<float, Kv8::INT8>(a, s);
}

}  // namespace gdr
