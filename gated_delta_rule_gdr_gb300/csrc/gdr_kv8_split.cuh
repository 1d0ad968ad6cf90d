// gdr_kv8_split.cuh -- attention over the 8-bit paged cache for few query rows a cached head
// (one token a request, a few drafted ones) and for fp32 queries (gdr_kv8_attn, gdr_kv8_attn_shared).
//
// Query i of a request (n queries, the last n of kv tokens) sees keys j <= kv - n + i:
//   x_j = scale ks (q . kcode_j) / ln 2,  o = sum_j p_j vs vcode_j / sum_j p_j,  p_j = 2^x_j
// with the scales ks, vs of j's page.  One pass: every row keeps a reference exponent M (a
// whole number, so that moving it rescales exactly) over x_j + log2 vs, and
//   P_j = 2^(x_j + log2 vs - M + 14),  O += P_j vcode_j,  l += P_j / vs,  o = O / l:
// the value scale rides in the exponent's addend and costs nothing per element.
//
// Bound: the cache's bytes.  Measured: 256 requests of 100 to 8192 keys, 8 heads a cached head
// (1029 MB) 0.166 ms = 6.2 TB/s, 91 % of the measured copy rate; one of a million keys (1074
// MB) 0.171 ms = 6.3 TB/s; loads alone took the million 0.167.  At group
// size 8 a byte of keys or values meets 16 flops, far
// below what the tensor cores need, so the kernel's job is to keep enough loads in flight
// and to stay within the issue slots: 12 warps an SM, each with two 8 KB slabs (32 tokens of
// keys and values) of its own coming by TMA, no barrier between warps inside an item.
// Both products are warp MMAs m16n8k16 on halves, transposed: S^T = K q^T and O^T = V^T P^T,
// so that the 16-row side of the MMA holds keys or value columns and the 8-column side the
// query rows: one token of up to 8 heads a cached head wastes nothing (with the rows on the
// 16-row side half of every product, exponential and register would be).  Codes of both
// types and normalised bf16 queries are exact in a half, weights keep 11 bits.  The codes go
// from the swizzled slab straight to A fragments:
//   keys    a lane reads D / 4 consecutive bytes of one key; which of the row's values a lane
//           holds is free as long as the query fragment is laid out alike
//   values  a lane reads D / 8 bytes of four tokens and interleaves them pairwise (PRMT); which
//           row of which MMA a value is, is free, and chosen so that a lane's outputs are
//           D / 8 consecutive values
// with every 16-byte load of a quarter warp on distinct banks under the 128-byte swizzle.
// The weights turn from accumulator to B layout by one 8 x 8 transpose (MOVM) per 8 keys.
// fp32 queries are split in two halves (22 bits), two MMAs for one; their weights in three bfloat16
// (24 bits), three for one, with the value codes as bfloat16: halves end at 2^-24, two of them as
// one, and beside a large weight without a value (its output is what the small ones give) two
// halves were off by 1.3e-4 at scores 20 nats below it.  64 decodes of 100 to 8000 keys: 71.3 us, with
// the two halves 63.4.

#pragma once

#include "gdr_kv8_attn.cuh"

#include <cmath>

namespace gdr {
namespace {

namespace sp {
constexpr int SLAB = 32;               // tokens a warp takes at a time
// An item is R blocks of 8 rows.  Four warps take the slabs of a unit in turn, each with a ring of
// its own, and join their sums at the item's end.
constexpr int NW = 4;                  // warps a CTA
constexpr int UT = NW * SLAB;          // tokens of a unit
// What an item's ends cost, in units (0 / 1 / 2 / 3: 256 requests of 100 to 8192 keys 0.179 / 0.172 /
// 0.166 / 0.166 ms, of 100 to 600 0.043 / 0.039 / 0.036 / 0.036).
constexpr int ITEM = 2;
// Slabs of a ring and CTAs an SM (two blocks' fragments need the registers of 8 warps an SM).
template <int R> constexpr int ST = R == 2 ? 3 : 2;
template <int R> constexpr int CPS = R == 2 ? 2 : 3;
template <int D> constexpr uint32_t SLAB_BYTES = SLAB * D;
template <int D> constexpr uint32_t STAGE = 2 * SLAB_BYTES<D>;     // keys, then values
template <int R, int D> constexpr uint32_t OFF_RED = NW * ST<R> * STAGE<D>;   // [4 warps][4 rows][D]
template <int R, int D> constexpr uint32_t OFF_SCAL = OFF_RED<R, D> + 4 * 4 * D * 4;
template <int R, int D> constexpr uint32_t SMEM = OFF_SCAL<R, D> + NW * ST<R> * 4 * 4;   // [ring][ST][2 groups][2]
}  // namespace sp

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two halves that are codes as bfloat16, exactly (8 bits hold either type's).
__device__ __forceinline__ uint32_t codes_bf(uint32_t h) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(x.x, x.y);
}
// The transpose of an 8 x 8 matrix of halves, a row's pair a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Byte offset of 16-byte chunk c of token t in a slab of tokens of D bytes stored in
// 128-byte rows under the 128-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t slab_offset(uint32_t t, uint32_t c) {
    const uint32_t row = D == 128 ? t : t >> 1, ch = D == 128 ? c : (t & 1) * 4 + c;
    return row * 128u + ((ch ^ (row & 7u)) << 4);
}

template <typename E, Kv8 KV, int D, int R, class A>
__global__ void __launch_bounds__(32 * sp::NW, sp::CPS<R>)
kv8_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const A a) {
    using sp::SLAB, sp::SLAB_BYTES, sp::STAGE, sp::NW, sp::UT;
    constexpr int ST = sp::ST<R>, RB = 8 * R;
    constexpr bool HL = sizeof(E) == 4;          // fp32: queries and weights in parts
    constexpr int NKS = D / 16, NVT = D / 16;    // k steps of K q^T, row tiles of O^T
    constexpr int LD = D / 4, LO = D / 8;        // values of a query, of an output row that a lane holds
    extern __shared__ __align__(1024) uint8_t sm[];
    __shared__ __align__(8) uint64_t s_bar[NW * ST];
    __shared__ FirstPlace<A> s_place;
    __shared__ int64_t s_scan[2 * NW];
    __shared__ float s_stat[2][NW][RB];          // M, l of each warp at an item's end
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    float *s_red = reinterpret_cast<float *>(sm + sp::OFF_RED<R, D>);
    float *s_scal = reinterpret_cast<float *>(sm + sp::OFF_SCAL<R, D>) + warp * ST * 4;
    const uint32_t stage0 = smem_u32(sm) + (uint32_t)warp * ST * STAGE<D>;
    auto bar = [&](int i) { return smem_u32(&s_bar[warp * ST + i]); };

    if (lane == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(bar(i), 1);
        fence_mbar_init();
        if (warp == 0) s_abort = 0;
    }
    if (tid == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    grid_dependency_wait();
    find_place<RB, UT, 32 * NW, sp::ITEM>(a, &s_place, s_scan);
    const int64_t u0 = s_place.u0;
    const int units = (int)(s_place.u1 - u0);
    if (units == 0) {
        if (tid == 0) a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
        grid_launch_dependents();
        return;
    }
    int4 entry = make_int4(-1, 0, 0, 0);
    const int P = 1 << a.page_log2;

    // ---- loads: lane i < 2 brings tokens 16 i .. 16 i + 15 of the slab, a page entry ahead
    using Cur = Cursor<RB, UT, A>;
    Cur ld;
    ld.start(a, s_place);
    int left = units, fill = 0;          // units to load, stage to fill
    int page = -1, page_h = 0;           // of the slab to be loaded next
    int pend = -1;                       // stage whose scales are on their way
    float pend_k = 0.f, pend_v = 0.f;
    auto look_up = [&]() {
        page = -1;
        if (lane < 2 && left > 0) {
            const int tok = ld.t * UT + warp * SLAB + 16 * lane;
            if (tok < ld.r.kv) page = a.table[table_at(a, ld.r, ld.s) + (tok >> a.page_log2)];
            page_h = ld.h;
        }
    };
    auto flush = [&]() {
        if (pend < 0) return;
        if (lane < 2) {
            s_scal[pend * 4 + lane * 2] = pend_k;
            s_scal[pend * 4 + lane * 2 + 1] = pend_v;
        }
        __syncwarp();
        pend = -1;
    };
    auto issue = [&]() {
        flush();
        if (left == 0) return;
        const bool there = lane < 2 && page >= 0 && page < a.N;
        const unsigned m = __ballot_sync(0xffffffffu, there);
        if (lane == 0) mbar_arrive_expect_tx(bar(fill), (uint32_t)__popc(m) * 32u * D);
        __syncwarp();
        pend_k = 0.f, pend_v = -1.f;     // a page that is gone
        if (there) {
            const int tok = ld.t * UT + warp * SLAB + 16 * lane;
            const int64_t ph = (int64_t)page * a.Hkv + page_h;
            const int row = (int)((ph << a.page_log2) + (tok & (P - 1)));
            const uint32_t dst = stage0 + (uint32_t)fill * STAGE<D> + (uint32_t)lane * 16 * D;
            tma_load_2d(dst, &tm_k, bar(fill), 0, D == 128 ? row : row >> 1);
            tma_load_2d(dst + SLAB_BYTES<D>, &tm_v, bar(fill), 0, D == 128 ? row : row >> 1);
            pend_k = a.ks[ph];
            pend_v = fminf(fmaxf(a.vs[ph], kv8::kVsMin), kv8::kVsMax);
        }
        pend = fill;
        fill = fill == ST - 1 ? 0 : fill + 1;
        --left;
        ld.next_unit(a);
        look_up();
    };
    // a limit of zero: the first wait has run out before it begins, whether its data is there or not
    bool ok = a.limit_ns != 0;
    look_up();
#pragma unroll 1
    for (int i = 0; i < ST; ++i) issue();
    __syncwarp();

    // ---- the items
    Cur c;
    c.start(a, s_place);
    int stage = 0;
    uint32_t phase = 0;
    int waited = 0;
#pragma unroll 1
    for (int done = 0, item = 0; done < units; ++item) {
        const int t_first = c.t, t_last = min(c.nt, t_first + units - done);   // this CTA's units of the item
        const int row0 = c.b * RB, rows = min(RB, c.r.n * a.G - row0);
        // query fragments: row 8 n + g, values LD t4 .. LD t4 + LD - 1, word j of a key holding
        // values 4 j .. 4 j + 3 of them
        uint32_t qf[HL ? 2 : 1][R][NKS][2];
        // of rows 8 n + 2 t4 + e: the score factor in units of ln 2, the keys seen, M and l
        float cs[R][2], M[R][2], l[R][2];
        int lim[R][2];
#pragma unroll
        for (int n = 0; n < R; ++n) {
            const int lr = 8 * n + g, at = row0 + lr;
            float f[LD];
            if (lr < rows) {
                const int i = at / a.G;
                const E *q = static_cast<const E *>(a.q) + (int64_t)(c.r.q0 + i) * a.q_stride +
                             (int64_t)(c.h * a.G + at - i * a.G) * D + t4 * LD;
#pragma unroll
                for (int v = 0; v < LD; v += Vec16<E>::N) Vec16<E>::load(q + v, f + v);
            } else {
#pragma unroll
                for (int v = 0; v < LD; ++v) f[v] = 0.f;
            }
            float amax = 0.f;
#pragma unroll
            for (int v = 0; v < LD; ++v) amax = fmaxf(amax, fabsf(f[v]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const float fac = row_factor(amax) * a.sign, csg = a.scale_log2 * fabsf(1.f / fac);
#pragma unroll
            for (int j = 0; j < NKS; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float x0 = f[4 * j + 2 * k] * fac, x1 = f[4 * j + 2 * k + 1] * fac;
                    qf[0][n][j][k] = pack_h2(x0, x1);
                    if constexpr (HL) {
                        const float2 h = __half22float2(*reinterpret_cast<__half2 *>(&qf[0][n][j][k]));
                        qf[HL ? 1 : 0][n][j][k] = pack_h2(x0 - h.x, x1 - h.y);
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r2 = 8 * n + 2 * t4 + e;
                cs[n][e] = __shfl_sync(0xffffffffu, csg, 4 * (2 * t4 + e));
                lim[n][e] = r2 < rows ? seen_by(a, c.r, (row0 + r2) / a.G) : 0;
                M[n][e] = -INFINITY;
                l[n][e] = 0.f;
            }
        }
        // the fewest keys that a row of the item sees: below them no mask is needed
        const int lim_all = seen_by(a, c.r, row0 / a.G);
        float o[R][NVT][4];     // value LO g + 2 j + (k >> 1) of row 8 n + 2 t4 + (k & 1)
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
            for (int j = 0; j < NVT; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][j][k] = 0.f;

#pragma unroll 1
        for (int t = t_first; t < t_last; ++t) {
            if (ok) {
                ok = mbar_test_wait(bar(stage), phase);
                if (!ok) ok = role_wait_slow(bar(stage), phase, a.limit_ns, &s_abort, false);
                ok = __all_sync(0xffffffffu, ok);
                waited += ok;
            }
            const uint32_t kb = stage0 + (uint32_t)stage * STAGE<D>, vb = kb + SLAB_BYTES<D>;
            const int tok0 = t * UT + warp * SLAB;
            if (ok && tok0 < c.end) {
                float ksc[2], vsc[2];      // of the slab's two groups of 16 tokens
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ksc[i] = s_scal[stage * 4 + 2 * i];
                    vsc[i] = s_scal[stage * 4 + 2 * i + 1];
                }
                const bool gone = vsc[0] < 0.f || vsc[1] < 0.f;
                // value codes of places without a cached token: zero, so that no stale NaN
                // meets a zero weight
                if (gone || tok0 + SLAB > c.r.kv) {
#pragma unroll 1
                    for (int x = lane; x < SLAB * D / 16; x += 32) {
                        const int tk = x / (D / 16);
                        if (tok0 + tk >= c.r.kv || vsc[tk >> 4] < 0.f)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             vb + slab_offset<D>(tk, x % (D / 16))), "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // scores of 32 keys: x[i][n][k] is key 16 i + g + 8 (k >> 1), row 8 n + 2 t4 + (k & 1)
                float x[2][R][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int n = 0; n < R; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[i][n][k] = 0.f;
#pragma unroll
                for (int v = 0; v < NKS / 4; ++v) {
                    uint32_t w[2][2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint4 u = lds128(kb + slab_offset<D>(16 * i + 8 * e + g, t4 * (NKS / 4) + v));
                            w[i][e][0] = u.x, w[i][e][1] = u.y, w[i][e][2] = u.z, w[i][e][3] = u.w;
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t f[4];
                            decode4_h<KV>(w[i][0][j], f[0], f[2]);
                            decode4_h<KV>(w[i][1][j], f[1], f[3]);
#pragma unroll
                            for (int n = 0; n < R; ++n) {
                                mma_f16(x[i][n], f, qf[0][n][4 * v + j][0], qf[0][n][4 * v + j][1]);
                                if constexpr (HL)
                                    mma_f16(x[i][n], f, qf[HL ? 1 : 0][n][4 * v + j][0], qf[HL ? 1 : 0][n][4 * v + j][1]);
                            }
                        }
                }
                if (gone || tok0 + SLAB > lim_all) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < R; ++n)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (tok0 + 16 * i + g + 8 * (k >> 1) >= lim[n][k & 1] || vsc[i] < 0.f) x[i][n][k] = -INFINITY;
                }
                // exponents are x cs ks + log2 vs; a factor of at least 2^-126 keeps masked scores
                // at -inf where a scale is zero
                float ev[2], iv[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ev[i] = vsc[i] < 0.f ? 0.f : __log2f(vsc[i]);
                    iv[i] = vsc[i] < 0.f ? 0.f : __frcp_rn(vsc[i]);
                }
                float kf[2][R][2], mx[R][2];
                bool grow = false;
#pragma unroll
                for (int n = 0; n < R; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[n][e] = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            kf[i][n][e] = fmaxf(cs[n][e] * ksc[i], 1.2e-38f);
                            mx[n][e] = fmaxf(mx[n][e], fmaf(fmaxf(x[i][n][e], x[i][n][2 + e]), kf[i][n][e], ev[i]));
                        }
                        grow |= mx[n][e] > M[n][e] + kv8::kTau;
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < R; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = mx[n][e];
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                            m = fmaxf(M[n][e], ceilf(m));
                            const float w = part_weight(M[n][e], m);
                            M[n][e] = m;
                            l[n][e] *= w;
#pragma unroll
                            for (int j = 0; j < NVT; ++j) {
                                o[n][j][e] *= w;
                                o[n][j][2 + e] *= w;
                            }
                        }
                }
                uint32_t pf[HL ? 3 : 1][2][R][2];     // weights of 16 keys as the B operand
#pragma unroll
                for (int n = 0; n < R; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float add = ev[i] - (M[n][e] == -INFINITY ? 0.f : M[n][e]) + kv8::kOff;
                            p[e] = ex2(fmaf(x[i][n][e], kf[i][n][e], add));
                            p[2 + e] = ex2(fmaf(x[i][n][2 + e], kf[i][n][e], add));
                            l[n][e] = fmaf(p[e] + p[2 + e], iv[i], l[n][e]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if constexpr (HL) {
                                float r0 = p[2 * k], r1 = p[2 * k + 1];
#pragma unroll
                                for (int w = 0; w < (HL ? 3 : 1); ++w) {
                                    const uint32_t b = pack_bf16x2(r0, r1);
                                    pf[w][i][n][k] = transpose8(b);
                                    r0 -= __uint_as_float(b << 16);
                                    r1 -= __uint_as_float(b & 0xffff0000u);
                                }
                            } else {
                                pf[0][i][n][k] = transpose8(pack_h2(p[2 * k], p[2 * k + 1]));
                            }
                        }
                    }
                // outputs: rows g and g + 8 of tile j are values LO g + 2 j and the next
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    constexpr int WPT = D / 32;    // words of a token that a lane reads
                    uint32_t w[4][WPT];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t tk = 16 * i + 2 * t4 + (k & 1) + 8 * (k >> 1);
                        if constexpr (D == 128) {
                            const uint4 u = lds128(vb + slab_offset<D>(tk, g));
                            w[k][0] = u.x, w[k][1] = u.y, w[k][WPT - 2] = u.z, w[k][WPT - 1] = u.w;
                        } else {
                            const uint2 u = lds64(vb + slab_offset<D>(tk, g >> 1) + (g & 1) * 8);
                            w[k][0] = u.x, w[k][1] = u.y;
                        }
                    }
#pragma unroll
                    for (int v = 0; v < WPT; ++v)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            uint32_t f[4];
                            decode4_h<KV>(__byte_perm(w[0][v], w[1][v], hf ? 0x7362 : 0x5140), f[0], f[1]);
                            decode4_h<KV>(__byte_perm(w[2][v], w[3][v], hf ? 0x7362 : 0x5140), f[2], f[3]);
                            if constexpr (HL) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) f[k] = codes_bf(f[k]);
#pragma unroll
                                for (int w = (HL ? 3 : 1) - 1; w >= 0; --w)
#pragma unroll
                                    for (int n = 0; n < R; ++n) mma_bf(o[n][2 * v + hf], f, pf[w][i][n][0], pf[w][i][n][1]);
                            } else {
#pragma unroll
                                for (int n = 0; n < R; ++n) mma_f16(o[n][2 * v + hf], f, pf[0][i][n][0], pf[0][i][n][1]);
                            }
                        }
                }
            }
            __syncwarp();
            if (ok) issue();
            if (++stage == ST) stage = 0, phase ^= 1;
        }

        // ---- the item's end: the four warps' sums joined
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
                if (g == 0) {
                    s_stat[0][warp][8 * n + 2 * t4 + e] = M[n][e];
                    s_stat[1][warp][8 * n + 2 * t4 + e] = l[n][e];
                }
            }
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
        const bool first = t_first == 0, last = t_last == c.nt;
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (first ? 1 : 0)) * RB;
        if (first && !last)
            entry = make_int4(cta_of(s_place, u0 + done + c.nt - 1, s_place.i0 + item), c.s, c.h, c.b);
#pragma unroll
        for (int pass = 0; pass < 2 * R; ++pass) {       // rows 4 pass .. 4 pass + 3
            if (4 * pass >= rows) break;
            if ((t4 >> 1) == (pass & 1)) {
                const int n = pass >> 1;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int lr = 8 * n + 2 * t4 + e;
                    float Mt = -INFINITY;
#pragma unroll
                    for (int w = 0; w < NW; ++w) Mt = fmaxf(Mt, s_stat[0][w][lr]);
                    const float f = M[n][e] == Mt ? 1.f : part_weight(M[n][e], Mt);
                    float *dst = s_red + (warp * 4 + (lr & 3)) * D;
#pragma unroll
                    for (int m = 0; m < LO / 4; ++m) {   // a lane's LO consecutive values, banks spread
                        const int ch = (LO / 4) * g + (m ^ ((g >> 1) & (LO / 4 - 1)));
                        *reinterpret_cast<float4 *>(dst + 4 * ch) =
                            make_float4(o[n][2 * m][e] * f, o[n][2 * m][2 + e] * f, o[n][2 * m + 1][e] * f,
                                        o[n][2 * m + 1][2 + e] * f);
                    }
                }
            }
            __syncthreads();
            // thread -> row 4 pass + tid / 32, values of lane
            {
                const int rr = tid >> 5, lr = 4 * pass + rr;
                if (lr < rows) {
                    float Mt = -INFINITY, L = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) Mt = fmaxf(Mt, s_stat[0][w][lr]);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float m = s_stat[0][w][lr];
                        L = fmaf(m == Mt ? 1.f : part_weight(m, Mt), s_stat[1][w][lr], L);
                    }
                    constexpr int VL = D / 32;       // consecutive values a lane writes
                    float y[VL];
                    const int ch4 = lane * VL / 4, gg = ch4 / (LO / 4), m = ch4 % (LO / 4);
                    const int ch = (LO / 4) * gg + (m ^ ((gg >> 1) & (LO / 4 - 1)));
#pragma unroll
                    for (int v = 0; v < VL; ++v) y[v] = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w)
#pragma unroll
                        for (int v = 0; v < VL; ++v)
                            y[v] += s_red[(w * 4 + rr) * D + 4 * ch + (lane * VL) % 4 + v];
                    if (first && last) {
                        const int at = c.b * RB + lr, i = at / a.G;
                        const int64_t row = (int64_t)(c.r.q0 + i) * a.Hq + c.h * a.G + (at - i * a.G);
                        if (complete_row<D>(a, c.r, row, lane * VL, lane == 0, y, Mt, L)) {
                            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                            for (int v = 0; v < VL; ++v) {
                                if constexpr (HL)
                                    static_cast<float *>(a.out)[row * D + lane * VL + v] = y[v] * inv;
                                else
                                    static_cast<__nv_bfloat16 *>(a.out)[row * D + lane * VL + v] =
                                        __float2bfloat16_rn(y[v] * inv);
                            }
                            if (a.lse && lane == 0)
                                a.lse[row] = L == 0.f ? -INFINITY
                                                      : ((Mt == -INFINITY ? 0.f : Mt) - kv8::kOff + log2f(L)) *
                                                            0.693147180559945f;
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < VL; ++v) a.part_o[(slot + lr) * D + lane * VL + v] = y[v];
                        if (lane == 0) {
                            a.part_ml[2 * (slot + lr)] = Mt;
                            a.part_ml[2 * (slot + lr) + 1] = L;
                        }
                    }
                }
            }
            __syncthreads();
        }
        done += t_last - t_first;
        c.next_of_item(a);
    }
    if (!ok) {   // leave no copy in flight
        if (a.limit_ns == 0 && lane == 0) atomicOr(&g_device_error_word, kDevErrTimeout);
        entry.x = -1;
        const int issued = units - left;
        for (int k = waited; k < issued; ++k) mbar_wait(bar(k % ST), (uint32_t)(k / ST) & 1u, kCleanupLimitNs);
    }
    if (tid == 0) a.entry[blockIdx.x] = entry;
    grid_launch_dependents();
}

// The cache as rows of 128 bytes; boxes of 16 tokens, 128-byte swizzle.
bool make_cache_map(CUtensorMap *m, const void *ptr, int64_t tokens, int D) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {128, (cuuint64_t)(tokens * D / 128)};
    cuuint64_t strides[1] = {128};
    cuuint32_t box[2] = {128, (cuuint32_t)(16 * D / 128)};
    cuuint32_t es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename E, Kv8 KV, int D, int R, class A>
cudaError_t launch_split_r(A &a, const void *kc, const void *vc, void *ws, int64_t rows, cudaStream_t s) {
    constexpr int RB = 8 * R;
    const int ctas = sp::CPS<R> * sm_count();
    place_parts(a, ws, ctas, RB);
    CUtensorMap mk, mv;
    const int64_t tokens = ((int64_t)a.N * a.Hkv) << a.page_log2;
    if (!make_cache_map(&mk, kc, tokens, D) || !make_cache_map(&mv, vc, tokens, D)) return cudaErrorInvalidValue;
    auto kernel = kv8_split_kernel<E, KV, D, R, A>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kernel, sp::SMEM<R, D>, allowed);
    if (e != cudaSuccess) return e;
    attended.store(true, std::memory_order_relaxed);
    if ((e = launch_after(kernel, dim3((unsigned)ctas), 32 * sp::NW, sp::SMEM<R, D>, s, mk, mv, a)) != cudaSuccess)
        return e;
    return launch_merge<E, D, RB>(a, rows, s);
}

// The item's shape by the most rows of a cached head that a request has.
enum class Shape { R8, R16, TILE };
Shape shape_of(int max_q, int G, Elem e) {
    const int64_t rows = (int64_t)max_q * G;
    if (rows <= 8) return Shape::R8;
    // fp32 (the accuracy path) stays at 16 rows: its fragments are twice as large.  bf16 up to 16
    // rows: 32 requests on 16 k keys 0.112 ms here, 0.136 in the tile kernel, 4 on 4000 keys 17.0
    // and 26.8 us (32 on 300 keys 21.3 and 20.2); beyond, 32 rows in warps of their own on shared
    // slabs took 0.243 ms against the tile kernel's 0.182 at the time (32 on 300 keys 22 us; 20.6
    // in the tile kernel since an item's ends count in the division)
    return rows <= 16 || e == Elem::F32 ? Shape::R16 : Shape::TILE;
}
template <typename E, Kv8 KV, int D, class A>
cudaError_t launch_split(A &a, Shape sh, const void *kc, const void *vc, void *ws, int64_t rows, cudaStream_t s) {
    return sh == Shape::R8 ? launch_split_r<E, KV, D, 1>(a, kc, vc, ws, rows, s)
                           : launch_split_r<E, KV, D, 2>(a, kc, vc, ws, rows, s);
}
template <class A>
cudaError_t launch_split_any(A &a, Shape sh, const void *k_cache, const void *v_cache, int D, Elem e, Kv8 kv, void *ws,
                             int64_t rows, cudaStream_t s) {
    const bool bf = e == Elem::BF16, f8 = kv == Kv8::E4M3;
    if (D == 128) {
        if (bf) return f8 ? launch_split<__nv_bfloat16, Kv8::E4M3, 128>(a, sh, k_cache, v_cache, ws, rows, s)
                          : launch_split<__nv_bfloat16, Kv8::INT8, 128>(a, sh, k_cache, v_cache, ws, rows, s);
        return f8 ? launch_split<float, Kv8::E4M3, 128>(a, sh, k_cache, v_cache, ws, rows, s)
                  : launch_split<float, Kv8::INT8, 128>(a, sh, k_cache, v_cache, ws, rows, s);
    }
    if (bf) return f8 ? launch_split<__nv_bfloat16, Kv8::E4M3, 64>(a, sh, k_cache, v_cache, ws, rows, s)
                      : launch_split<__nv_bfloat16, Kv8::INT8, 64>(a, sh, k_cache, v_cache, ws, rows, s);
    return f8 ? launch_split<float, Kv8::E4M3, 64>(a, sh, k_cache, v_cache, ws, rows, s)
              : launch_split<float, Kv8::INT8, 64>(a, sh, k_cache, v_cache, ws, rows, s);
}
size_t shape_workspace_bytes(Shape sh, int D) {
    const int sms = sm_count();
    switch (sh) {
        case Shape::R8: return part_bytes(sp::CPS<1> * sms, 8, D);
        case Shape::R16: return part_bytes(sp::CPS<2> * sms, 16, D);
        case Shape::TILE: break;
    }
    return part_bytes(sms, kKv8TileRows, D);
}

}  // namespace
}  // namespace gdr
