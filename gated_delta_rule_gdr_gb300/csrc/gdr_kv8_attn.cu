// gdr_kv8_attn.cu -- attention over the 8-bit paged cache for few query rows a cached head
// (one token a request, a few drafted ones) and for fp32 queries (gdr_kv8_attn).
//
// Query i of a request (n queries, the last n of kv tokens) sees keys j <= kv - n + i:
//   x_j = scale ks (q . kcode_j) / ln 2,  o = sum_j p_j vs vcode_j / sum_j p_j,  p_j = 2^x_j
// with the scales ks, vs of j's page.  One pass: every row keeps a reference exponent M (a
// whole number, so that moving it rescales exactly) over x_j + log2 vs, and
//   P_j = 2^(x_j + log2 vs - M + 7),  O += P_j vcode_j,  l += P_j / vs,  o = O / l:
// the value scale rides in the exponent's addend and costs nothing per element.
//
// Bound: the cache's bytes.  At group size 8 a byte of keys or values meets 16 flops, far
// below what the tensor cores need, so the kernel's job is to keep enough loads in flight
// and to stay within the issue slots: 8 warps an SM, each with three 8 KB slabs (32 tokens
// of keys and values) of its own coming by TMA, no barrier between warps inside an item.
// Both products are warp MMAs m16n8k16 on halves: codes of both types and normalised bf16
// queries are exact in a half, weights keep 11 bits.  The 16 rows of the MMA are the rows of
// one item; the codes go from the swizzled slab straight to B fragments:
//   keys    a lane reads 32 consecutive bytes of one key; which of the row's values a lane
//           holds is free as long as the query fragment is laid out alike
//   values  a lane reads 16 bytes of four tokens and interleaves them pairwise (PRMT); which
//           column of which MMA a value is, is free, and chosen so that a lane's outputs are
//           D / 4 consecutive values
// with every 16-byte load of a quarter warp on distinct banks under the 128-byte swizzle.
// fp32 queries and their weights are split in two halves each (22 bits), two MMAs for one.

#include "gdr_kv8_attn.cuh"

#include <cmath>

namespace gdr {
namespace {

namespace sp {
constexpr int NW = 4, NT = 32 * NW;    // warps a CTA; two CTAs an SM
constexpr int SLAB = 32;               // tokens a warp takes at a time
constexpr int UT = SLAB * NW;          // a unit: one slab for each warp
constexpr int ST = 3;                  // slabs a warp has in flight
constexpr int RB = 16;                 // rows of an item
template <int D> constexpr uint32_t SLAB_BYTES = SLAB * D;
template <int D> constexpr uint32_t STAGE = 2 * SLAB_BYTES<D>;     // keys, then values
template <int D> constexpr uint32_t OFF_RED = NW * ST * STAGE<D>;  // [4 warps][4 rows][D] floats
template <int D> constexpr uint32_t OFF_SCAL = OFF_RED<D> + NW * 4 * D * 4;   // [NW][ST][2 groups][2]
template <int D> constexpr uint32_t SMEM = OFF_SCAL<D> + NW * ST * 4 * 4 + 1024;
}  // namespace sp

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <typename E, Kv8 KV, int D>
__global__ void __launch_bounds__(sp::NT, 2)
kv8_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const AttnArgs a) {
    using namespace sp;
    constexpr bool HL = sizeof(E) == 4;          // two halves for queries and weights
    constexpr int NKS = D / 16, NVT = D / 8;     // k steps of q.k, column tiles of the output
    constexpr int LD = D / 4;                    // values of a row that a lane holds
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t s_bar[NW * ST];
    __shared__ Place s_place;
    __shared__ int64_t s_scan[NW];
    __shared__ float s_stat[2][NW][RB];          // M, l of each warp at an item's end
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    float *s_red = reinterpret_cast<float *>(sm + OFF_RED<D>);
    float *s_scal = reinterpret_cast<float *>(sm + OFF_SCAL<D>) + warp * ST * 4;
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
    find_place<RB, UT, NT>(a, &s_place, s_scan);
    const int64_t u0 = s_place.u0, total = s_place.total;
    const int units = (int)(s_place.u1 - u0);
    if (units == 0) {
        if (tid == 0) a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
        grid_launch_dependents();
        return;
    }
    int4 entry = make_int4(-1, 0, 0, 0);
    const int P = 1 << a.page_log2;

    // ---- loads: lane i < 2 brings tokens 16 i .. 16 i + 15 of the slab, a page entry ahead
    using Cur = Cursor<RB, UT>;
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
            if (tok < ld.r.kv) page = a.table[(int64_t)ld.s * a.W + (tok >> a.page_log2)];
            page_h = ld.h;
        }
    };
    auto issue = [&]() {
        if (lane < 2 && pend >= 0) {
            s_scal[pend * 4 + lane * 2] = pend_k;
            s_scal[pend * 4 + lane * 2 + 1] = pend_v;
        }
        pend = -1;
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
    look_up();
#pragma unroll 1
    for (int i = 0; i < ST; ++i) issue();
    __syncwarp();

    // ---- the items
    Cur c;
    c.start(a, s_place);
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    int waited = 0;
#pragma unroll 1
    for (int done = 0; done < units;) {
        const int t_first = c.t, t_last = min(c.nt, t_first + units - done);   // this CTA's units of the item
        const int rows = min(RB, c.r.n * a.G - c.b * RB);
        // query fragments: rows g and g + 8, values LD t4 .. LD t4 + LD - 1, word j of a key
        // holding values 4 j .. 4 j + 3 of them
        uint32_t qf[HL ? 2 : 1][NKS][4];
        float cs[2];                       // score factor of the row, in units of ln 2
        int lim[2];                        // keys it sees
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int lr = g + 8 * e, at = c.b * RB + lr;
            float f[LD];
            lim[e] = 0;
            if (lr < rows) {
                const int i = at / a.G;
                const E *q = static_cast<const E *>(a.q) + (int64_t)(c.r.q0 + i) * a.q_stride +
                             (int64_t)(c.h * a.G + at - i * a.G) * D + t4 * LD;
#pragma unroll
                for (int v = 0; v < LD; v += Vec16<E>::N) Vec16<E>::load(q + v, f + v);
                lim[e] = seen_by(c.r, i);
            } else {
#pragma unroll
                for (int v = 0; v < LD; ++v) f[v] = 0.f;
            }
            float amax = 0.f;
#pragma unroll
            for (int v = 0; v < LD; ++v) amax = fmaxf(amax, fabsf(f[v]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const float fac = row_factor(amax) * a.sign;
            cs[e] = a.scale_log2 * fabsf(1.f / fac);
#pragma unroll
            for (int j = 0; j < NKS; ++j) {
                const float x0 = f[4 * j] * fac, x1 = f[4 * j + 1] * fac, x2 = f[4 * j + 2] * fac, x3 = f[4 * j + 3] * fac;
                qf[0][j][e] = pack_h2(x0, x1);
                qf[0][j][2 + e] = pack_h2(x2, x3);
                if constexpr (HL) {
                    const float2 h0 = __half22float2(*reinterpret_cast<__half2 *>(&qf[0][j][e]));
                    const float2 h1 = __half22float2(*reinterpret_cast<__half2 *>(&qf[0][j][2 + e]));
                    qf[HL ? 1 : 0][j][e] = pack_h2(x0 - h0.x, x1 - h0.y);
                    qf[HL ? 1 : 0][j][2 + e] = pack_h2(x2 - h1.x, x3 - h1.y);
                }
            }
        }
        // the fewest keys that a row of the item sees: below them no mask is needed
        const int lim_all = seen_by(c.r, c.b * RB / a.G);
        float o[NVT][4];
#pragma unroll
        for (int j = 0; j < NVT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

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
            float ksc[2], vsc[2];
            bool gone = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ksc[i] = s_scal[stage * 4 + 2 * i];
                vsc[i] = s_scal[stage * 4 + 2 * i + 1];
                gone |= vsc[i] < 0.f;
            }
            if (ok && tok0 < c.end) {
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
                // scores of 32 keys: column n of tile i is key 8 i + n
                float x[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
                    uint32_t w[NKS];
#pragma unroll
                    for (int v = 0; v < NKS / 4; ++v) {
                        const uint4 u = lds128(kb + slab_offset<D>(8 * i + g, t4 * (NKS / 4) + v));
                        w[4 * v] = u.x, w[4 * v + 1] = u.y, w[4 * v + 2] = u.z, w[4 * v + 3] = u.w;
                    }
#pragma unroll
                    for (int j = 0; j < NKS; ++j) {
                        const uint32_t b0 = decode2_h<KV>(w[j] & 0xffffu), b1 = decode2_h<KV>(w[j] >> 16);
                        mma_f16(x[i], qf[0][j], b0, b1);
                        if constexpr (HL) mma_f16(x[i], qf[HL ? 1 : 0][j], b0, b1);
                    }
                }
                // exponents y = x cs ks + log2 vs of both rows, masked where needed
                float kf[2][2], ev[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ev[i] = vsc[i] < 0.f ? 0.f : __log2f(vsc[i]);
                    kf[0][i] = cs[0] * ksc[i];
                    kf[1][i] = cs[1] * ksc[i];
                }
                if (gone || tok0 + SLAB > lim_all) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tk = tok0 + 8 * i + 2 * t4 + (e & 1);
                            if (tk >= lim[e >> 1] || vsc[i >> 1] < 0.f) x[i][e] = __int_as_float(0xff800000);
                        }
                }
                float mx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        m[i] = fmaxf(fmaxf(x[2 * i][2 * e], x[2 * i][2 * e + 1]),
                                     fmaxf(x[2 * i + 1][2 * e], x[2 * i + 1][2 * e + 1]));
                    mx[e] = fmaxf(m[0] == -INFINITY ? -INFINITY : fmaf(m[0], kf[e][0], ev[0]),
                                  m[1] == -INFINITY ? -INFINITY : fmaf(m[1], kf[e][1], ev[1]));
                }
                if (__any_sync(0xffffffffu, mx[0] > M[0] + kv8::kTau || mx[1] > M[1] + kv8::kTau)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = mx[e];
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                        m = fmaxf(M[e], ceilf(m));
                        const float w = part_weight(M[e], m);
                        M[e] = m;
                        l[e] *= w;
#pragma unroll
                        for (int j = 0; j < NVT; ++j) {
                            o[j][2 * e] *= w;
                            o[j][2 * e + 1] *= w;
                        }
                    }
                }
                uint32_t pf[HL ? 2 : 1][2][4];     // weights of 16 keys as the A operand
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = M[e] == -INFINITY ? 0.f : M[e];
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const float add = ev[kk] - ref + kv8::kOff;
                        float p[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float s = x[2 * kk + (k >> 1)][2 * e + (k & 1)];
                            p[k] = s == -INFINITY ? 0.f : ex2(fmaf(s, kf[e][kk], add));
                        }
                        l[e] = fmaf((p[0] + p[1]) + (p[2] + p[3]), vsc[kk] < 0.f ? 0.f : 1.f / vsc[kk], l[e]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t hi = pack_h2(p[2 * k], p[2 * k + 1]);
                            pf[0][kk][2 * k + e] = hi;
                            if constexpr (HL) {
                                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                                pf[HL ? 1 : 0][kk][2 * k + e] = pack_h2(p[2 * k] - h.x, p[2 * k + 1] - h.y);
                            }
                        }
                    }
                }
                // outputs: column n of tile j is value (D / 8) n + j
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    constexpr int WPT = D / 32;    // words of a token that a lane reads
                    uint32_t w[4][WPT];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t tk = 16 * kk + 2 * t4 + (k & 1) + 8 * (k >> 1);
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
                            const uint32_t lo = __byte_perm(w[0][v], w[1][v], hf ? 0x7362 : 0x5140);
                            const uint32_t hi = __byte_perm(w[2][v], w[3][v], hf ? 0x7362 : 0x5140);
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const int j = 4 * v + 2 * hf + z;
                                const uint32_t b0 = decode2_h<KV>(z ? lo >> 16 : lo & 0xffffu);
                                const uint32_t b1 = decode2_h<KV>(z ? hi >> 16 : hi & 0xffffu);
                                mma_f16(o[j], pf[0][kk], b0, b1);
                                if constexpr (HL) mma_f16(o[j], pf[HL ? 1 : 0][kk], b0, b1);
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
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (t4 == 0) {
                s_stat[0][warp][g + 8 * e] = M[e];
                s_stat[1][warp][g + 8 * e] = l[e];
            }
        }
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
        const bool first = t_first == 0, last = t_last == c.nt;
        const int64_t slot = ((int64_t)blockIdx.x * 2 + (first ? 1 : 0)) * RB;
        if (first && !last)
            entry = make_int4(cta_of(u0 + done + c.nt - 1, total, s_place.ctas), c.s, c.h, c.b);
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {       // rows 4 pass .. 4 pass + 3
            if (4 * pass >= rows) break;
            const int e = pass >> 1;
            if ((g >> 2) == (pass & 1)) {
                const int lr = g + 8 * e;
                float Mt = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w) Mt = fmaxf(Mt, s_stat[0][w][lr]);
                const float f = M[e] == Mt ? 1.f : part_weight(M[e], Mt);
                float *dst = s_red + (warp * 4 + (g & 3)) * D;
#pragma unroll
                for (int m = 0; m < LD / 4; ++m) {   // a lane's LD consecutive values, banks spread
                    float4 u;
                    float *uf = reinterpret_cast<float *>(&u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int d = 4 * m + k, n2 = d / NVT, j = d % NVT;   // column 2 t4 + n2 of tile j
                        uf[k] = (e ? o[j][2 + n2] : o[j][n2]) * f;
                    }
                    const int ch = (LD / 4) * t4 + (m ^ ((2 * t4 + g) & (LD / 4 - 1)));
                    *reinterpret_cast<float4 *>(dst + 4 * ch) = u;
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
                    const int ch4 = lane * VL / 4, tt = ch4 / (LD / 4), m = ch4 % (LD / 4);
                    const int ch = (LD / 4) * tt + (m ^ ((2 * tt + lr) & (LD / 4 - 1)));
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

template <typename E, Kv8 KV, int D>
cudaError_t launch_split(const AttnArgs &a, const void *kc, const void *vc, int ctas, int rows, cudaStream_t s) {
    CUtensorMap mk, mv;
    const int64_t tokens = ((int64_t)a.N * a.Hkv) << a.page_log2;
    if (!make_cache_map(&mk, kc, tokens, D) || !make_cache_map(&mv, vc, tokens, D)) return cudaErrorInvalidValue;
    auto kernel = kv8_split_kernel<E, KV, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sp::SMEM<D>);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)ctas, sp::NT, sp::SMEM<D>, s>>>(mk, mv, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_merge<E, D, sp::RB, 8>(a, ctas, rows, s);
}

}  // namespace

// Rows of a cached head that the split kernel takes; bf16 with more goes to the tile kernel.
// At 16 rows the split kernel's MMAs are full; beyond, it reads the cache once for every 16
// rows (5 drafted tokens x 8 heads on 16 k keys 0.42 ms against 0.33 ms here, a chunk of 1000
// tokens on 65 k 7.3 ms against 1.5 ms).
bool kv8_tiles(int max_q, int G, Elem e) { return e == Elem::BF16 && (int64_t)max_q * G > sp::RB; }

size_t kv8_attn_workspace_bytes(int, int max_q, int, int Hq, int Hkv, int D, Elem e) {
    return kv8_tiles(max_q, Hq / Hkv, e) ? part_bytes(sm_count(), kKv8TileRows, D)
                                         : part_bytes(2 * sm_count(), sp::RB, D);
}

cudaError_t launch_kv8_attn(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, const int *table,
                            const int *kv_len, const int *cu_q, float scale, void *out, float *lse, int S,
                            int max_q, int total_q, int Hq, int Hkv, int D, int W, int page, int N, Elem e,
                            Kv8 kv, void *ws, cudaStream_t s) {
    if (kv8_tiles(max_q, Hq / Hkv, e))
        return launch_kv8_tile(q, q_stride, k_cache, v_cache, k_scale, v_scale, table, kv_len, cu_q, scale, out,
                               lse, S, max_q, total_q, Hq, Hkv, D, W, page, N, kv, ws, s);
    const int ctas = 2 * sm_count();
    AttnArgs a{};
    a.q = q, a.q_stride = q_stride, a.ks = k_scale, a.vs = v_scale, a.table = table, a.kv_len = kv_len;
    a.cu_q = cu_q, a.scale_log2 = fabsf(scale) * 1.4426950408889634f, a.sign = scale < 0.f ? -1.f : 1.f;
    a.out = out, a.lse = lse;
    place_parts(a, ws, ctas, sp::RB);
    a.S = S, a.total_q = total_q, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.W = W, a.N = N;
    a.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    a.limit_ns = wait_limit_ns();
    const int64_t rows64 = (int64_t)max_q * a.G;
    const int rows = rows64 > sp::RB ? sp::RB : (int)rows64;
    const bool bf = e == Elem::BF16, f8 = kv == Kv8::E4M3;
    if (D == 128) {
        if (bf) return f8 ? launch_split<__nv_bfloat16, Kv8::E4M3, 128>(a, k_cache, v_cache, ctas, rows, s)
                          : launch_split<__nv_bfloat16, Kv8::INT8, 128>(a, k_cache, v_cache, ctas, rows, s);
        return f8 ? launch_split<float, Kv8::E4M3, 128>(a, k_cache, v_cache, ctas, rows, s)
                  : launch_split<float, Kv8::INT8, 128>(a, k_cache, v_cache, ctas, rows, s);
    }
    if (bf) return f8 ? launch_split<__nv_bfloat16, Kv8::E4M3, 64>(a, k_cache, v_cache, ctas, rows, s)
                      : launch_split<__nv_bfloat16, Kv8::INT8, 64>(a, k_cache, v_cache, ctas, rows, s);
    return f8 ? launch_split<float, Kv8::E4M3, 64>(a, k_cache, v_cache, ctas, rows, s)
              : launch_split<float, Kv8::INT8, 64>(a, k_cache, v_cache, ctas, rows, s);
}

cudaError_t take_kv8_split_error_word(unsigned *value) { return take_error_word(value); }

}  // namespace gdr
