// gdr_norm_rope.cu -- norms of queries and keys for each head with the rotation by the token's
// position in the same pass (gdr_qk_norm_rope), and its backward (gdr_qk_norm_rope_bwd).
//
// Of a head's D values x, with weights w and the rotation R of the token's position p:
//   r = (|x|^2 / N + eps)^-1/2  (N = D: root mean square, N = 1: unit length; or r = 1)
//   y = R(p) (w x r)
// R turns `rot / 2` pairs of values, pair i by the angle p f_i.  Backward, with g = R(p)^T dy:
//   dw = sum over tokens and heads of g x r,   dx = r (w g - x r^2 <w g, x> / N)
//
// Angles.  A position may be any 31-bit number, so p f_i passes what fp32 resolves.  f_i enters as
// a 64-bit fixed-point fraction of a turn, F = frac(f_i / 2 pi) 2^64: p F modulo 2^64 is p f_i
// without its whole turns, exactly but for F's own rounding (2^-64 turns times p), and costs
// three integer multiplications a token and pair, shared by the token's heads.
//
// Work.  A head's values are taken by D / 16 lanes, 16 values each in chunks of 16 bytes: chunks that
// a pair lies across (or within), so that no value changes lanes but in the row's sums, and
// neighbouring lanes have neighbouring chunks.  A warp takes 32 / (D / 16) rows (a token's head) at once: a
// pass.  The rows of a tensor, heads in tokens in order, are divided evenly among the warps of the CTAs that
// the tensor got, queries and keys by their cost.  A lane copies its chunks asynchronously to a
// place of its own in shared memory, ST - 1 passes ahead, so that no registers wait for memory and
// nothing synchronises.
//
// Bound: bytes (forward 2, backward 3 times the tensors).  Measured, 16384 tokens, 32 + 8 heads of
// 128 bf16 values out of one projection, weights and rotation: forward (336 MB, 50 us at the
// measured copy rate) 56 us, backward with the weights' gradients (503 MB, 75 us) 82 us; in fp32 106 and
// 163 us; 65536 tokens of 64 heads to unit length (2147 MB, 322 us) 326 us, of 1 + 1 heads with rotation
// (67 MB) 16 us, of 8 + 8 heads of 64 values (268 MB) 51 us: a token's sines and cosines then serve one
// pass.  Rings of 2, 3 and 4 passes: 65, 56 and 58 us bf16, 105, 113 and 114 fp32.  With the values in
// registers, four passes' (forward) or two (backward) in flight: 60 and 98 us (the backward's spill).

#include "gdr_launch.cuh"

#include <algorithm>

namespace gdr {
namespace {

namespace nr {
constexpr int NT = 256, NW = NT / 32;
// CTAs an SM, passes of a warp's ring.  Without rotation or gradients three bf16 CTAs have the registers
// (4096 tokens of 32 heads to unit length, from the L2, 7.8 us against 9.4; 65536 of 64 330 against 332; in
// fp32 16384 of 32 heads 87 against 83).
template <typename E, int ROT, bool BWD> constexpr int CPS = sizeof(E) == 2 && ROT == 0 && !BWD ? 3 : 2;
template <typename E, int ROT, bool BWD> constexpr int ST = sizeof(E) == 4 || CPS<E, ROT, BWD> == 3 ? 2 : 3;
template <typename E> constexpr int NC = sizeof(E);               // chunks of a lane's 16 values
template <typename E, bool BWD> constexpr uint32_t STAGE = (BWD ? 2 : 1) * NC<E> * 512;   // bytes of a warp's pass
constexpr int RUN = 4;         // passes of a warp where there are few
}

struct NormTensor {
    const void *x, *g;       // input; gradient of the output (backward)
    void *y;                 // output; gradient of the input (backward)
    int64_t xs, gs, ys;      // elements between tokens
    const float *w;          // [D] or null
    float *part;             // backward: [CTAs of the tensor][D] sums of the weights' gradient, or null
    int H;
};
struct NormArgs {
    NormTensor t[2];         // queries, keys
    const int *positions;
    const double *freq;
    float eps, inv_n;
    int T, dlog2, rot, split;    // split: CTAs of the first tensor
    bool norm;
};

// A chunk: brought to the lane's place in shared memory (none: zeros), taken from there as packed pairs of
// floats, stored.
__device__ __forceinline__ void bring_chunk(uint32_t dst, const void *src, bool has) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(has ? 16 : 0) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t src, uint64_t &a, uint64_t &b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(src) : "memory");
}
template <typename E> struct Chunk;
template <> struct Chunk<float> {
    static __device__ __forceinline__ void get(uint32_t src, uint64_t *f) { lds128(src, f[0], f[1]); }
    static __device__ __forceinline__ void store(float *p, const uint64_t *f) {
        *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(f[0], f[1]);
    }
};
template <> struct Chunk<__nv_bfloat16> {
    static __device__ __forceinline__ void get(uint32_t src, uint64_t *f) {
        uint64_t u[2];
        lds128(src, u[0], u[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = (uint32_t)(u[i >> 1] >> (32 * (i & 1)));
            f[i] = f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const uint64_t *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(f[i], a, b);
            w[i] = pack_bf16x2(a, b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
// Where in a row the chunks of a lane (of `lanes` a row) begin, and a lane's packed pair e.  With pairs (i, i +
// rot / 2) the first rot / 16 lanes have what is turned, a chunk of the second half for each of the first.
template <typename E> struct Places {
    static constexpr int NC = nr::NC<E>, CV = 16 / NC;       // values of a chunk
    int at[NC];
    __device__ __forceinline__ Places(int j, int lanes, int rot, bool halves) {
        const int t = rot >> 4;                              // lanes of the turned part
        if (halves && j < t) {
#pragma unroll
            for (int c = 0; c < NC; ++c) at[c] = CV * (j + t * (c % (NC / 2))) + (c < NC / 2 ? 0 : rot / 2);
        } else {
            const int from = halves ? rot : 0, n = halves ? lanes - t : lanes;
#pragma unroll
            for (int c = 0; c < NC; ++c) at[c] = from + CV * (j - (halves ? t : 0) + n * c);
        }
    }
    __device__ __forceinline__ int pair(int e) const { return at[e / (8 / NC)] + 2 * (e % (8 / NC)); }
};

// frac(f / 2 pi) 2^64.  1 / (2 pi) in two doubles, so that F is good to its last bits.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    constexpr double c = 0.15915494309189535, c_lo = -9.839338337591243e-18;
    const double t = f * c, t_lo = fma(f, c, -t) + f * c_lo;
    double x = t - floor(t);
    x = x < 1.0 ? x : 0.0;
    return (uint64_t)(x * 18446744073709551616.0) + (uint64_t)(int64_t)(t_lo * 18446744073709551616.0);
}
// Sine and cosine of a 32-bit fraction of a turn.  bf16: the hardware's approximations (absolute error
// 2^-20, a rounding is 2^-8 of a value).  fp32: the quarter turn is taken off while the angle is
// an integer, so that what remains converts to 2^-25 of an eighth of a turn.
template <typename E>
__device__ __forceinline__ void turn_sincos(uint32_t hi, float &s, float &c) {
    if constexpr (sizeof(E) == 4) {
        const uint32_t q = (hi + 0x20000000u) >> 30;
        float s0, c0;
        sincospif((float)(int)(hi - (q << 30)) * 4.656612873077393e-10f, &s0, &c0);   // 2^-31
        s = q & 1 ? c0 : s0;
        c = q & 1 ? -s0 : c0;
        if (q & 2) s = -s, c = -c;
    } else {
        __sincosf((float)(int)hi * 1.4629180792671596e-9f, &s, &c);                   // pi 2^-31
    }
}
template <typename E>
__device__ __forceinline__ float inverse_root(float x) {
    if constexpr (sizeof(E) == 4) return 1.f / sqrtf(x);
    return rsqrtf(x);
}

// The rotation of a lane's pairs.  ROT 1: pairs (i, i + rot / 2), packed pairs e and e + 4, two of them an
// instruction; ROT 2: pairs (2 i, 2 i + 1).
template <typename E, int ROT>
struct Turn {
    static constexpr int NC = nr::NC<E>;
    float c[8], s[8];
    bool on[NC];          // which chunks are turned (ROT 1: all or none)
    __device__ __forceinline__ Turn(const Places<E> &p, int rot) {
#pragma unroll
        for (int i = 0; i < NC; ++i) on[i] = p.at[i] < rot;
    }
    __device__ __forceinline__ void set(const uint64_t *f, const Places<E> &pl, uint32_t p) {
        if constexpr (ROT == 1) {
            if (on[0])
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    turn_sincos<E>((uint32_t)((f[pl.pair(e >> 1) + (e & 1)] * (uint64_t)p) >> 32), s[e], c[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (on[e / (8 / NC)]) turn_sincos<E>((uint32_t)((f[pl.pair(e) >> 1] * (uint64_t)p) >> 32), s[e], c[e]);
        }
    }
    template <bool BACK>
    __device__ __forceinline__ void apply(uint64_t (&f)[8]) const {
        if constexpr (ROT == 1) {
            if (on[0])
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t a = f[e], b = f[e + 4], minus = 0x8000000080000000ull;
                    const uint64_t c2 = f2_pack(c[2 * e], c[2 * e + 1]), s2 = f2_pack(s[2 * e], s[2 * e + 1]);
                    f[e] = f2_fma(BACK ? b : b ^ minus, s2, f2_mul(a, c2));
                    f[e + 4] = f2_fma(BACK ? a ^ minus : a, s2, f2_mul(b, c2));
                }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (on[e / (8 / NC)]) {
                    float a, b;
                    f2_unpack(f[e], a, b);
                    const float sn = BACK ? -s[e] : s[e];
                    f[e] = f2_pack(fmaf(-b, sn, a * c[e]), fmaf(a, sn, b * c[e]));
                }
        }
    }
};
template <typename E> struct Turn<E, 0> {
    __device__ __forceinline__ Turn(const Places<E> &, int) {}
};

// The sum of a packed pair over the lanes of a head.  LOG: log2 of these lanes, or -1: `log`.
template <int LOG>
__device__ __forceinline__ float head_sum(uint64_t v, int log) {
    float a, b;
    f2_unpack(v, a, b);
    a += b;
    if constexpr (LOG >= 0) {
#pragma unroll
        for (int off = 1; off < (1 << LOG); off <<= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    } else {
        for (int off = 1; off < (1 << log); off <<= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    }
    return a;
}
__device__ __forceinline__ uint64_t dot8(const uint64_t (&a)[8], const uint64_t (&b)[8]) {
    uint64_t v = f2_mul(a[0], b[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) v = f2_fma(a[e], b[e], v);
    return v;
}

// ROT: 0 no rotation, 1 pairs (i, i + rot / 2), 2 pairs (2 i, 2 i + 1).  LOG: log2 of D / 16, or -1:
// any.  BWD: the backward; DW: and the weights' gradients.
template <typename E, int ROT, int LOG, bool BWD, bool DW>
__global__ void __launch_bounds__(nr::NT, (nr::CPS<E, ROT, BWD>)) norm_rope_kernel(const NormArgs a) {
    using nr::NT, nr::NW;
    constexpr int NC = nr::NC<E>, ST = nr::ST<E, ROT, BWD>;
    constexpr uint32_t STAGE = nr::STAGE<E, BWD>;
    constexpr bool WSM = BWD && DW && ROT != 0;      // the weights in shared memory: registers are short
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ uint64_t s_f[ROT ? 256 : 1];
    __shared__ __align__(16) float s_w[WSM ? 512 : 4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int which = (int)blockIdx.x >= a.split;
    const int cta = which ? blockIdx.x - a.split : blockIdx.x, ctas = which ? gridDim.x - a.split : a.split;
    const NormTensor t = a.t[which];
    const int plog2 = LOG >= 0 ? LOG : a.dlog2 - 4, D = 16 << plog2;
    const int j = lane & ((1 << plog2) - 1), grp = lane >> plog2, HB = 32 >> plog2;
    const Places<E> at(j, 1 << plog2, a.rot, ROT == 1);

    // a warp's run of passes; this lane's row of the pass that is brought next, and of the one that is
    // computed next: token, head, and where the row begins
    const int H = t.H;
    const int64_t all = ((int64_t)a.T * H + HB - 1) >> (5 - plog2), nw = (int64_t)ctas * NW, gw = (int64_t)cta * NW + warp;
    const int64_t first = all * gw / nw, row = (first << (5 - plog2)) + grp;
    const int left = (int)(all * (gw + 1) / nw - first);
    const int at_t = HB / H, at_h = HB - at_t * H;           // a pass on
    int tok = (int)(row / H), h = (int)(row - (int64_t)tok * H), tok_b = tok, h_b = h;
    const int64_t in_row = (int64_t)h << a.dlog2;
    const E *xr = static_cast<const E *>(t.x) + tok * t.xs + in_row;
    const E *gr = BWD ? static_cast<const E *>(t.g) + tok * t.gs + in_row : nullptr;
    E *yr = static_cast<E *>(t.y) + tok * t.ys + in_row;
    auto next_row = [&](int &tk, int &hd) {                  // true: past the token's last head
        tk += at_t, hd += at_h;
        const bool past = hd >= H;
        if (past) hd -= H, ++tk;
        return past;
    };
    auto move = [&](auto *&p, int64_t stride, bool past) { p += at_t * stride + (at_h << a.dlog2) + (past ? stride - ((int64_t)H << a.dlog2) : 0); };
    const uint32_t ring = smem_u32(sm) + (uint32_t)warp * ST * STAGE + 16u * lane;
    int brought = 0;
    uint32_t fill = 0;
    auto bring = [&]() {
        if (brought < left) {
            const bool has = tok_b < a.T;                    // the last pass may have fewer rows
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                bring_chunk(ring + fill + 512u * c, has ? xr + at.at[c] : t.x, has);
                if constexpr (BWD) bring_chunk(ring + fill + 512u * (NC + c), has ? gr + at.at[c] : t.g, has);
            }
            const bool past = next_row(tok_b, h_b);
            move(xr, t.xs, past);
            if constexpr (BWD) move(gr, t.gs, past);
            ++brought;
        }
        fill = fill == (ST - 1) * STAGE ? 0 : fill + STAGE;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto position = [&](int tk) { return a.positions ? a.positions[min(tk, a.T - 1)] : 0; };

    grid_dependency_wait();
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) bring();
    int p_next = left > 0 ? position(tok) : 0;
    if constexpr (ROT != 0)
        for (int i = tid; i < a.rot / 2; i += NT) s_f[i] = turn_fraction(a.freq[i]);
    uint64_t w[8];
    if constexpr (WSM) {
        for (int i = tid; i < D; i += NT) s_w[i] = t.w ? t.w[i] : 1.f;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = t.w ? f2_pack(t.w[at.pair(e)], t.w[at.pair(e) + 1]) : f2_pack(1.f, 1.f);
    }
    if constexpr (ROT != 0) __syncthreads();
    uint64_t dw[DW ? 8 : 1];
    if constexpr (DW) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = 0;
    }

    Turn<E, ROT> turn(at, a.rot);
    int turned = -1;                  // the token that `turn` is for
    uint32_t stage = 0;
#pragma unroll 1
    for (int k = 0; k < left; ++k) {
        asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
        uint64_t f[8], d[BWD ? 8 : 1];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            Chunk<E>::get(ring + stage + 512u * c, f + 8 / NC * c);
            if constexpr (BWD) Chunk<E>::get(ring + stage + 512u * (NC + c), d + 8 / NC * c);
        }
        stage = stage == (ST - 1) * STAGE ? 0 : stage + STAGE;
        bring();          // into the place that was read in the pass before
        const int p = p_next, here = tok;
        const bool has = here < a.T, live = has && p >= 0;   // p < 0: not a token, no output and a gradient of zero
        const bool past = next_row(tok, h);
        p_next = position(tok);
        if constexpr (ROT != 0)
            if (here != turned) {
                turn.set(s_f, at, (uint32_t)p);
                turned = here;
            }
        float r = 1.f;
        if (a.norm) r = inverse_root<E>(fmaf(head_sum<LOG>(dot8(f, f), plog2), a.inv_n, a.eps));
        const uint64_t r2 = f2_pack(r, r);
        if constexpr (!BWD) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f2_mul(f2_mul(f[e], r2), w[e]);
            if constexpr (ROT != 0) turn.template apply<false>(f);
        } else {
            if constexpr (ROT != 0) turn.template apply<true>(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f2_mul(f[e], r2);          // x r
            if constexpr (DW) {
                if (live) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[e] = f2_fma(d[e], f[e], dw[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                if constexpr (WSM) lds128(smem_u32(s_w + at.pair(e)), w[e], w[e + 1]);
                d[e] = f2_mul(d[e], w[e]), d[e + 1] = f2_mul(d[e + 1], w[e + 1]);
            }
            if (a.norm) {
                const float dot = -head_sum<LOG>(dot8(d, f), plog2) * a.inv_n;
                const uint64_t k2 = f2_pack(dot, dot);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = f2_mul(r2, f2_fma(f[e], k2, d[e]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = d[e];
            }
            if (!live)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = 0;
        }
        if (BWD ? has : live)
#pragma unroll
            for (int c = 0; c < NC; ++c) Chunk<E>::store(yr + at.at[c], f + 8 / NC * c);
        move(yr, t.ys, past);
    }
    if constexpr (DW) {
        // lanes with the same values, then the warps, in a fixed order
        float d[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) f2_unpack(dw[e], d[2 * e], d[2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            for (int off = 1 << plog2; off < 32; off <<= 1) d[e] += __shfl_xor_sync(0xffffffffu, d[e], off);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        static_assert(ST * STAGE >= 512 * sizeof(float) && ST >= 2, "");
        float *s_dw = reinterpret_cast<float *>(sm);      // [NW][D], over the rings
        if (grp == 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) s_dw[warp * D + at.pair(e >> 1) + (e & 1)] = d[e];
        __syncthreads();
        for (int i = tid; i < D; i += NT) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) s += s_dw[k * D + i];
            if (t.part) t.part[(int64_t)cta * D + i] = s;
        }
    }
    grid_launch_dependents();
}

// The weights' gradients from the CTAs' sums, of queries (blockIdx.x 0) and keys: a CTA for 32 of the
// D values, a lane for one, the 32 warps for every 32nd CTA's each.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const NormArgs a, int ctas, float *dwq, float *dwk) {
    __shared__ float s_sum[32][33];
    const int D = 1 << a.dlog2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = 32 * blockIdx.y + lane;
    grid_dependency_wait();
    float *dst = blockIdx.x ? dwk : dwq;
    const float *part = a.t[blockIdx.x].part;
    const int n = blockIdx.x ? ctas - a.split : a.split;
    if (dst) {
        float sum = 0.f;
#pragma unroll 4
        for (int c = warp; c < n; c += 32) sum += col < D ? part[((int64_t)c << a.dlog2) + col] : 0.f;
        s_sum[warp][lane] = sum;
        __syncthreads();
        sum = s_sum[lane][warp];           // value 32 blockIdx.y + warp, lane's part
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0 && 32 * blockIdx.y + warp < D) dst[32 * blockIdx.y + warp] = sum;
    }
    grid_launch_dependents();
}

// CTAs of both tensors: a warp for every RUN passes while the device has them, else all that are
// resident, in proportion to the passes and (the sines and cosines) half a pass for each that begins
// tokens.
int divide(NormArgs &a, int per_sm) {
    const int HB = 32 >> (a.dlog2 - 4);
    int64_t passes[2], want[2], cost[2];      // without the half pass 59 us for 32 + 8 heads, 56 with it
    for (int i = 0; i < 2; ++i) {
        passes[i] = ((int64_t)a.T * a.t[i].H + HB - 1) / HB;
        want[i] = (passes[i] + nr::RUN * nr::NW - 1) / (nr::RUN * nr::NW);
        cost[i] = 2 * passes[i] + (a.rot ? std::min(passes[i], (int64_t)a.T) : 0);
    }
    const int most = per_sm * sm_count();
    if (want[0] + want[1] <= most) {
        a.split = (int)want[0];
        return (int)(want[0] + want[1]);
    }
    int q = (int)((most * cost[0] + (cost[0] + cost[1]) / 2) / (cost[0] + cost[1]));
    if (passes[0] && q < 1) q = 1;
    if (passes[1] && q > most - 1) q = most - 1;
    a.split = q;
    return most;
}

template <typename E, int ROT, int LOG, bool BWD, bool DW>
cudaError_t launch_norm_k(NormArgs &a, float *dwq, float *dwk, float *ws, cudaStream_t s) {
    const int ctas = divide(a, nr::CPS<E, ROT, BWD>);
    if (DW) {
        a.t[0].part = ws;
        a.t[1].part = ws + ((size_t)a.split << a.dlog2);
    }
    if (ctas > 0) {
        constexpr size_t smem = (size_t)nr::NW * nr::ST<E, ROT, BWD> * nr::STAGE<E, BWD>;
        auto kernel = norm_rope_kernel<E, ROT, LOG, BWD, DW>;
        static std::atomic<uint64_t> allowed{0};
        cudaError_t e = allow_smem(kernel, smem, allowed);
        if (e != cudaSuccess) return e;
        if ((e = launch_after(kernel, dim3((unsigned)ctas), nr::NT, smem, s, a)) != cudaSuccess) return e;
    }
    if constexpr (DW)
        return launch_after(norm_weight_grad_kernel, dim3(2, ((1u << a.dlog2) + 31) / 32), 1024, 0, s, a, ctas, dwq, dwk);
    return cudaSuccess;
}
template <typename E, int ROT, int LOG>
cudaError_t launch_norm_d(NormArgs &a, bool bwd, float *dwq, float *dwk, float *ws, cudaStream_t s) {
    if (!bwd) return launch_norm_k<E, ROT, LOG, false, false>(a, nullptr, nullptr, nullptr, s);
    if (dwq || dwk) return launch_norm_k<E, ROT, LOG, true, true>(a, dwq, dwk, ws, s);
    return launch_norm_k<E, ROT, LOG, true, false>(a, nullptr, nullptr, nullptr, s);
}
template <typename E, int ROT>
cudaError_t launch_norm_r(NormArgs &a, bool bwd, float *dwq, float *dwk, float *ws, cudaStream_t s) {
    return a.dlog2 == 7   ? launch_norm_d<E, ROT, 3>(a, bwd, dwq, dwk, ws, s)
           : a.dlog2 == 6 ? launch_norm_d<E, ROT, 2>(a, bwd, dwq, dwk, ws, s)
                          : launch_norm_d<E, ROT, -1>(a, bwd, dwq, dwk, ws, s);
}
template <typename E>
cudaError_t launch_norm_e(NormArgs &a, int pairs, bool bwd, float *dwq, float *dwk, float *ws, cudaStream_t s) {
    if (a.rot == 0) return launch_norm_r<E, 0>(a, bwd, dwq, dwk, ws, s);
    return pairs == 0 ? launch_norm_r<E, 1>(a, bwd, dwq, dwk, ws, s) : launch_norm_r<E, 2>(a, bwd, dwq, dwk, ws, s);
}
NormArgs norm_args(const NormCall &c) {
    NormArgs a{};
    a.positions = c.positions, a.freq = c.freq;
    a.eps = c.eps, a.inv_n = c.mean ? 1.f / c.D : 1.f, a.norm = c.norm;
    a.T = c.T, a.rot = c.rot;
    while ((1 << a.dlog2) < c.D) ++a.dlog2;
    for (int i = 0; i < 2; ++i) {
        const NormCall::Tensor &t = c.t[i];
        a.t[i] = NormTensor{t.x, t.g, t.y, t.x_stride, t.g_stride, t.y_stride, t.w, nullptr, t.H};
    }
    return a;
}

}  // namespace

size_t norm_rope_workspace_bytes(int D) { return (size_t)nr::CPS<float, 0, true> * sm_count() * D * sizeof(float); }

cudaError_t launch_norm_rope(const NormCall &c, bool bwd, float *dwq, float *dwk, void *ws, Elem e, cudaStream_t s) {
    NormArgs a = norm_args(c);
    float *parts = static_cast<float *>(ws);
    return e == Elem::F32 ? launch_norm_e<float>(a, c.pairs, bwd, dwq, dwk, parts, s)
                          : launch_norm_e<__nv_bfloat16>(a, c.pairs, bwd, dwq, dwk, parts, s);
}

}  // namespace gdr
