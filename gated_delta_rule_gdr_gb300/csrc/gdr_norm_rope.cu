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
// Work.  A head's values are taken by D / 16 lanes, 16 values each in two pieces of 8: pieces
// that a pair lies across (or within), so that no value changes lanes but in the row's sums.
// A warp takes 32 / (D / 16) heads at once, U times over for loads in flight: a unit.  The units of
// a tensor, tokens in order, are divided evenly among the warps of the CTAs that the tensor
// got, queries and keys in proportion.
//
// Bound: bytes (forward 2, backward 3 times the tensors).

#include "gdr_launch.cuh"

namespace gdr {
namespace {

namespace nr {
constexpr int NT = 256, NW = NT / 32;
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

// 8 values of a piece, as they come and as floats.
template <typename E> struct Piece;
template <> struct Piece<float> {
    uint4 u[2];
    __device__ __forceinline__ void load(const float *p) {
        u[0] = *reinterpret_cast<const uint4 *>(p);
        u[1] = *reinterpret_cast<const uint4 *>(p + 4);
    }
    __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(u[i].x), f[4 * i + 1] = __uint_as_float(u[i].y);
            f[4 * i + 2] = __uint_as_float(u[i].z), f[4 * i + 3] = __uint_as_float(u[i].w);
        }
    }
    static __device__ __forceinline__ void store(float *p, const float *f) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <> struct Piece<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *f) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                   pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// frac(f / 2 pi) 2^64.  1 / (2 pi) in two doubles, so that F is good to its last bits.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    constexpr double c = 0.15915494309189535, c_lo = -9.839338337591978e-18;
    const double t = f * c, t_lo = fma(f, c, -t) + f * c_lo;
    double x = t - floor(t);
    x = x < 1.0 ? x : 0.0;
    return (uint64_t)(x * 18446744073709551616.0) + (uint64_t)(int64_t)(t_lo * 18446744073709551616.0);
}
// Sine and cosine of a 32-bit fraction of a turn.  bf16: the hardware's approximations (absolute error
// 2^-20, a rounding is 2^-9 of a value).  fp32: the quarter turn is taken off while the angle is
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

// ROT: 0 no rotation, 1 pairs (i, i + rot / 2), 2 pairs (2 i, 2 i + 1).
template <int ROT>
__device__ __forceinline__ void rotate(float (&f)[16], const float (&cs)[8], const float (&sn)[8], float sign, bool turned) {
    if (ROT == 0 || !turned) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = ROT == 1 ? i : 2 * i, ib = ROT == 1 ? i + 8 : 2 * i + 1;
        const float a = f[ia], b = f[ib], s = sn[i] * sign;
        f[ia] = fmaf(a, cs[i], -b * s);
        f[ib] = fmaf(a, s, b * cs[i]);
    }
}

// U: passes of a unit, whose loads are in flight together.  BWD: the backward; DW: and the weights'
// gradients.
template <typename E, int ROT, bool BWD, bool DW, int U>
__global__ void __launch_bounds__(nr::NT, 2) norm_rope_kernel(const NormArgs a) {
    using nr::NT, nr::NW;
    __shared__ uint64_t s_f[ROT ? 256 : 1];
    __shared__ float s_dw[DW ? NW : 1][DW ? 512 : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int which = (int)blockIdx.x >= a.split;
    const int cta = which ? blockIdx.x - a.split : blockIdx.x, ctas = which ? gridDim.x - a.split : a.split;
    const NormTensor t = a.t[which];
    const int plog2 = a.dlog2 - 4, j = lane & ((1 << plog2) - 1), grp = lane >> plog2, HB = 32 >> plog2;
    // the two pieces; a lane's pairs are 8 j .. 8 j + 7
    const int lanes_turned = a.rot >> 4;
    const bool turned = ROT != 0 && j < lanes_turned;
    const int p0 = ROT == 1 ? (turned ? j : 2 * j) : 2 * j, p1 = ROT == 1 && turned ? j + lanes_turned : p0 + 1;

    grid_dependency_wait();
    if constexpr (ROT != 0) {
        for (int i = tid; i < a.rot / 2; i += NT) s_f[i] = turn_fraction(a.freq[i]);
        __syncthreads();
    }
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = t.w ? t.w[8 * (i < 8 ? p0 : p1) + (i & 7)] : 1.f;
    float dw[DW ? 16 : 1];
    if constexpr (DW)
#pragma unroll
        for (int i = 0; i < 16; ++i) dw[i] = 0.f;

    const int passes = (t.H + HB - 1) / HB, chunks = (passes + U - 1) / U;
    const int64_t units = (int64_t)a.T * chunks, nw = (int64_t)ctas * NW, gw = (int64_t)cta * NW + warp;
    const int64_t u0 = units * gw / nw, u1 = units * (gw + 1) / nw;
    int64_t tok = chunks ? u0 / chunks : 0;
    int c = (int)(u0 - tok * chunks);
    float cs[8] = {}, sn[8] = {};
    int p = 0;
    bool fresh = true;
#pragma unroll 1
    for (int64_t u = u0; u < u1; ++u) {
        Piece<E> x[U][2], g[BWD ? U : 1][2];
        const E *xr = static_cast<const E *>(t.x) + tok * t.xs;
        const E *gr = BWD ? static_cast<const E *>(t.g) + tok * t.gs : nullptr;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = (c * U + i) * HB + grp;
            if (h < t.H) {
                const int at = h << a.dlog2;
                x[i][0].load(xr + at + 8 * p0);
                x[i][1].load(xr + at + 8 * p1);
                if constexpr (BWD) {
                    g[i][0].load(gr + at + 8 * p0);
                    g[i][1].load(gr + at + 8 * p1);
                }
            } else {
                x[i][0].zero(), x[i][1].zero();
                if constexpr (BWD) g[i][0].zero(), g[i][1].zero();
            }
        }
        if (fresh && a.positions) {
            p = a.positions[tok];
            if constexpr (ROT != 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (turned) turn_sincos<E>((uint32_t)((s_f[8 * j + i] * (uint64_t)(uint32_t)p) >> 32), sn[i], cs[i]);
                }
            }
        }
        fresh = false;
        E *yr = static_cast<E *>(t.y) + tok * t.ys;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = (c * U + i) * HB + grp, at = h << a.dlog2;
            float f[16];
            if (p < 0) {          // not a token: no output, and a gradient of zero (the warp's lanes agree)
                if (BWD && h < t.H) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = 0.f;
                    Piece<E>::store(yr + at + 8 * p0, f);
                    Piece<E>::store(yr + at + 8 * p1, f);
                }
                continue;
            }
            x[i][0].get(f), x[i][1].get(f + 8);
            float r = 1.f;
            if (a.norm) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
                for (int off = 1; off < (1 << plog2); off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                r = inverse_root<E>(fmaf(ss, a.inv_n, a.eps));
            }
            if constexpr (!BWD) {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] *= r * w[e];
                rotate<ROT>(f, cs, sn, 1.f, turned);
            } else {
                float d[16];
                g[i][0].get(d), g[i][1].get(d + 8);
                rotate<ROT>(d, cs, sn, -1.f, turned);
                if constexpr (DW)
                    if (h < t.H)
#pragma unroll
                        for (int e = 0; e < 16; ++e) dw[e] = fmaf(d[e], f[e] * r, dw[e]);
#pragma unroll
                for (int e = 0; e < 16; ++e) d[e] *= w[e];
                if (a.norm) {
                    float dot = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) dot = fmaf(d[e], f[e], dot);
                    for (int off = 1; off < (1 << plog2); off <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
                    const float k = -dot * a.inv_n * r * r;
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = r * fmaf(f[e], k, d[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = d[e];
                }
            }
            if (h < t.H) {
                Piece<E>::store(yr + at + 8 * p0, f);
                Piece<E>::store(yr + at + 8 * p1, f + 8);
            }
        }
        if (++c == chunks) c = 0, ++tok, fresh = true;
    }
    if constexpr (DW) {
        // lanes with the same values, then the warps, in a fixed order
#pragma unroll
        for (int e = 0; e < 16; ++e)
            for (int off = 1 << plog2; off < 32; off <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], off);
        if (grp == 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) s_dw[warp][8 * (e < 8 ? p0 : p1) + (e & 7)] = dw[e];
        __syncthreads();
        for (int i = tid; i < 1 << a.dlog2; i += NT) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NW; ++k) s += s_dw[k][i];
            if (t.part) t.part[((int64_t)cta << a.dlog2) + i] = s;
        }
    }
    grid_launch_dependents();
}

// The weights' gradients from the CTAs' sums: a CTA for queries and one for keys.
constexpr int SUM_NT = 1024;
__global__ void __launch_bounds__(SUM_NT) norm_weight_grad_kernel(const NormArgs a, int ctas, float *dwq, float *dwk) {
    __shared__ float s_sum[SUM_NT];
    const int D = 1 << a.dlog2, i = threadIdx.x & (D - 1), s = threadIdx.x >> a.dlog2, ns = SUM_NT >> a.dlog2;
    grid_dependency_wait();
    float *dst = blockIdx.x ? dwk : dwq;
    const float *part = a.t[blockIdx.x].part;
    const int n = blockIdx.x ? ctas - a.split : a.split;
    if (dst) {
        float sum = 0.f;
#pragma unroll 4
        for (int c = s; c < n; c += ns) sum += part[((int64_t)c << a.dlog2) + i];
        s_sum[threadIdx.x] = sum;
        __syncthreads();
        if (s == 0) {
            for (int k = 1; k < ns; ++k) sum += s_sum[k * D + i];
            dst[i] = sum;
        }
    }
    grid_launch_dependents();
}

constexpr int CTAS_PER_SM = 2;
int most_ctas() { return CTAS_PER_SM * sm_count(); }

// CTAs of both tensors: a warp for every unit while the device has them, else all that are resident,
// in proportion to the passes.
template <int U>
int divide(NormArgs &a) {
    const int HB = 32 >> (a.dlog2 - 4);
    int64_t units[2], passes[2];
    for (int i = 0; i < 2; ++i) {
        passes[i] = (a.t[i].H + HB - 1) / HB;
        units[i] = (passes[i] + U - 1) / U * a.T;
    }
    const int most = most_ctas();
    const int64_t want[2] = {(units[0] + nr::NW - 1) / nr::NW, (units[1] + nr::NW - 1) / nr::NW};
    if (want[0] + want[1] <= most) {
        a.split = (int)want[0];
        return (int)(want[0] + want[1]);
    }
    int q = (int)((most * passes[0] + (passes[0] + passes[1]) / 2) / (passes[0] + passes[1]));
    if (passes[0] && q < 1) q = 1;
    if (passes[1] && q > most - 1) q = most - 1;
    a.split = q;
    return most;
}

template <typename E, int ROT, bool BWD, bool DW, int U>
cudaError_t launch_norm_u(NormArgs &a, float *dwq, float *dwk, float *ws, cudaStream_t s) {
    const int ctas = divide<U>(a);
    if (DW) {
        a.t[0].part = ws;
        a.t[1].part = ws + ((size_t)a.split << a.dlog2);
    }
    if (ctas > 0) {
        cudaError_t e = launch_after(norm_rope_kernel<E, ROT, BWD, DW, U>, dim3((unsigned)ctas), nr::NT, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    if constexpr (DW)
        return launch_after(norm_weight_grad_kernel, dim3(2), SUM_NT, 0, s, a, ctas, dwq, dwk);
    return cudaSuccess;
}
template <typename E, int ROT>
cudaError_t launch_norm_r(NormArgs &a, bool bwd, float *dwq, float *dwk, float *ws, cudaStream_t s) {
    constexpr int U = sizeof(E) == 4 ? 2 : 4;
    if (!bwd) return launch_norm_u<E, ROT, false, false, U>(a, nullptr, nullptr, nullptr, s);
    if (dwq || dwk) return launch_norm_u<E, ROT, true, true, U / 2>(a, dwq, dwk, ws, s);
    return launch_norm_u<E, ROT, true, false, U / 2>(a, nullptr, nullptr, nullptr, s);
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

size_t norm_rope_workspace_bytes(int D) { return (size_t)most_ctas() * D * sizeof(float); }

cudaError_t launch_norm_rope(const NormCall &c, bool bwd, float *dwq, float *dwk, void *ws, Elem e, cudaStream_t s) {
    NormArgs a = norm_args(c);
    float *parts = static_cast<float *>(ws);
    return e == Elem::F32 ? launch_norm_e<float>(a, c.pairs, bwd, dwq, dwk, parts, s)
                          : launch_norm_e<__nv_bfloat16>(a, c.pairs, bwd, dwq, dwk, parts, s);
}

}  // namespace gdr
