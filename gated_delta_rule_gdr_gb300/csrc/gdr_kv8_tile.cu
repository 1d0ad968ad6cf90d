// gdr_kv8_tile.cu -- attention over the 8-bit paged cache for many bf16 query rows a cached
// head: prompts, chunks of prompts against a long cache, drafted tokens (gdr_kv8_attn).
//
// The same mathematics as the split kernel's (gdr_kv8_attn.cu): with a whole-number reference
// exponent M for each row over x_j + log2 vs,
//   P_j = 2^(x_j + log2 vs - M + 7),  O += P_j vcode_j,  l += P_j / vs,  o = O / l.
//
// Bound: the two products, 4 rows keys D flops, on the 5th-generation tensor cores.  An item
// is two tiles of 128 rows (row = query x group of heads) that share every key, a unit 128
// keys.  A tile's scores S (128 x 128 fp32) and sums O live in TMEM; its weights go back over
// S as halves and are the A operand of the second product from there, so that they never
// touch shared memory.  While the softmax of one tile runs, the products of the other do.
// The codes come by bulk copies (a page's block of a head is contiguous) and are widened to
// halves in the tensor core's swizzled layout: keys K-major, values MN-major from the same
// [token][64 values] rows, so values need no transpose.
//
// Warps: 0 loads (page entries and scales looked up one unit ahead), 1 issues the products
// and owns the TMEM, 4-7 widen, 8-11 and 12-15 the softmax of tile 0 and 1, a thread a row:
// maxima and sums never leave the thread.  Rings: 4 raw slots and 3 widened ones, each taking
// keys and values in turn.  No barrier spans the CTA inside the loop; every wait is bounded.

#include "gdr_kv8_attn.cuh"

#include <cmath>

namespace gdr {
namespace {

namespace tl {
constexpr int NT = 512;
constexpr int RB = kKv8TileRows, TR = 128, UT = 128;   // rows of an item and a tile, keys of a unit
constexpr int NRAW = 4, NCV = 3, NSC = 4;              // raw slots, widened slots, scale slots
template <int D> constexpr uint32_t RAW = UT * D;                    // a raw slot
template <int D> constexpr uint32_t CV = UT * D * 2;                 // a widened slot
constexpr uint32_t SLAB = 128 * 128;                                 // 128 rows x 64 halves
template <int D> constexpr uint32_t OFF_Q = 0;                       // two tiles
template <int D> constexpr uint32_t OFF_CV = 2 * TR * D * 2;
template <int D> constexpr uint32_t OFF_RAW = OFF_CV<D> + NCV * CV<D>;
template <int D> constexpr uint32_t OFF_SC = OFF_RAW<D> + NRAW * RAW<D>;   // [NSC][8 groups]{ks, vs, log2 vs, 1/vs}
template <int D> constexpr uint32_t SMEM = OFF_SC<D> + NSC * 8 * 16 + 1024;
static_assert(SMEM<128> + 512 <= 232448, "exceeds 227 KB of shared memory per CTA");
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;              // tile t at + 128 t
enum : int {
    B_RAWFULL = 0, B_RAWFREE = B_RAWFULL + NRAW, B_CVFULL = B_RAWFREE + NRAW, B_CVFREE = B_CVFULL + NCV,
    B_SC = B_CVFREE + NCV, B_Q = B_SC + NSC, B_S = B_Q + 2, B_P = B_S + 2, B_O = B_P + 2, B_DRAIN = B_O + 2,
    NUM_BARS = B_DRAIN + 1
};
}  // namespace tl

// Instruction descriptor of kind::f16 with half A and B and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

template <Kv8 KV, int D>
__global__ void __launch_bounds__(tl::NT, 1) kv8_tile_kernel(const AttnArgs a) {
    using namespace tl;
    using Cur = Cursor<RB, UT>;
    constexpr int NSL = D / 64;            // slabs of 64 values
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    __shared__ __align__(8) uint64_t s_bar[NUM_BARS];
    __shared__ Place s_place;
    __shared__ int64_t s_scan[NT / 32];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return smem_u32(&s_bar[i]); };
    float4 *s_sc = reinterpret_cast<float4 *>(sm + OFF_SC<D>);
    const int P = 1 << a.page_log2;

    if (tid == 0) {
        for (int i = 0; i < NRAW; ++i) {
            mbar_init(bar(B_RAWFULL + i), 1);
            mbar_init(bar(B_RAWFREE + i), 4);
        }
        for (int i = 0; i < NCV; ++i) {
            mbar_init(bar(B_CVFULL + i), 4);
            mbar_init(bar(B_CVFREE + i), 1);
        }
        for (int i = 0; i < NSC; ++i) mbar_init(bar(B_SC + i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_Q + i), 4);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_DRAIN), 1);
        s_abort = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();
    find_place<RB, UT, NT>(a, &s_place, s_scan);
    const int64_t u0 = s_place.u0;
    const int units = (int)(s_place.u1 - u0);
    if (units == 0) {
        if (tid == 0) a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
        grid_launch_dependents();
        return;
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](int b, uint32_t parity) { return role_wait(bar(b), parity & 1u, a.limit_ns, &s_abort); };
    auto warp_wait = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
    auto tiles_of = [&](const Cur &c) { return c.r.n * a.G - c.b * RB > TR ? 2 : 1; };

    if (warp == 0) {
        // ================================================================ loads
        // Lane i < 8 has keys 16 i .. 16 i + 15 of the unit; the first lane of a page copies it.
        Cur c;
        c.start(a, s_place);
        int page = -1;
        auto look_up = [&]() {
            page = -1;
            const int tok = c.t * UT + 16 * lane;
            if (lane < 8 && tok < c.r.kv) page = a.table[(int64_t)c.s * a.W + (tok >> a.page_log2)];
        };
        look_up();
        bool ok = true;
        int x = 0, pend = -1;
        float pk = 0.f, pv = 0.f;
        auto publish = [&]() {     // the scales of a unit, once they are here
            if (pend < 0) return;
            if (lane < 8)
                s_sc[(pend % NSC) * 8 + lane] = pv < 0.f ? make_float4(0.f, -1.f, 0.f, 0.f)
                                                         : make_float4(pk, pv, log2f(pv), 1.f / pv);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_SC + pend % NSC));
            pend = -1;
        };
#pragma unroll 1
        for (int k = 0; k < units; ++k) {
            const bool there = lane < 8 && page >= 0 && page < a.N;
            const int tok = c.t * UT + 16 * lane;
            const bool leader = there && (tok & (P - 1)) == 0;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, leader)) * (uint32_t)(P * D);
            const int64_t ph = (int64_t)page * a.Hkv + c.h;
            publish();
#pragma unroll 1
            for (int w = 0; w < 2; ++w, ++x) {      // keys, values
                const int sl = x % NRAW;
                if (x >= NRAW && !(ok = warp_wait(B_RAWFREE + sl, (uint32_t)(x / NRAW - 1)))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(B_RAWFULL + sl), bytes);
                __syncwarp();
                if (leader)
                    bulk_load(sb + OFF_RAW<D> + (uint32_t)sl * RAW<D> + (uint32_t)(16 * lane * D),
                              (w ? a.vc : a.kc) + (ph << a.page_log2) * D, (uint32_t)(P * D), bar(B_RAWFULL + sl));
            }
            if (!ok) break;
            pk = 0.f, pv = -1.f;     // a page that is gone
            if (there) {
                pk = a.ks[ph];
                pv = fminf(fmaxf(a.vs[ph], kv8::kVsMin), kv8::kVsMax);
            }
            pend = k;
            c.next_unit(a);
            if (k + 1 < units) look_up();
        }
        if (ok) publish();
        if (s_abort && lane == 0)    // leave no copy in flight
            for (int y = max(0, x - NRAW); y < x; ++y)
                mbar_wait(bar(B_RAWFULL + y % NRAW), (uint32_t)(y / NRAW) & 1u, kCleanupLimitNs);
    } else if (warp == 1) {
        // ================================================================ products
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_f16(TR, UT, false), id_o = idesc_f16(TR, D, true);
            Cur c, n;                // the unit whose second product is next, and the one after it
            c.start(a, s_place);
            n = c;
            bool ok = true, issued = false;
            uint32_t nq[2] = {0, 0}, np[2] = {0, 0};   // items and units that tile t has begun
            auto cv = [&](int x) { return sb + OFF_CV<D> + (uint32_t)(x % NCV) * CV<D>; };
            // scores of tile t for unit k (widened slot 2 k), n being its cursor
            auto scores = [&](int t, int k, bool new_item) {
                if (new_item) ok = ok && wait(B_Q + t, nq[t]++);
                ok = ok && wait(B_CVFULL + (2 * k) % NCV, (uint32_t)(2 * k / NCV));
                if (!ok) return;
                tc_fence_after();
                const uint64_t dq = sdesc_sw128(sb + OFF_Q<D> + (uint32_t)t * NSL * SLAB, 16, 1024);
                const uint64_t dk = sdesc_sw128(cv(2 * k), 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (uint32_t)(kk >> 2) * SLAB + (uint32_t)(kk & 3) * 32;
                    mma_bf16(tmem + TM_S + 128u * t, sdesc_add(dq, off), sdesc_add(dk, off), id_s, kk > 0);
                }
                mma_commit(bar(B_S + t));
                issued = true;
            };
            const int nt0 = tiles_of(n);
            for (int t = 0; t < nt0; ++t) scores(t, 0, true);
            if (ok) mma_commit(bar(B_CVFREE + 0));
#pragma unroll 1
            for (int k = 0; ok && k < units; ++k) {
                const int ntc = tiles_of(c);
                const bool last = c.t + 1 == c.nt || k + 1 == units, first = c.t == 0 || k == 0;
                bool fresh = false;
                int ntn = 0;
                if (k + 1 < units) {
                    n.next_unit(a);
                    fresh = n.t == 0;
                    ntn = tiles_of(n);
                }
#pragma unroll 1
                for (int t = 0; t < 2 && ok; ++t) {
                    if (t < ntc) {
                        ok = wait(B_P + t, np[t]++) && wait(B_CVFULL + (2 * k + 1) % NCV, (uint32_t)((2 * k + 1) / NCV));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t dv = sdesc_sw128(cv(2 * k + 1), SLAB, 1024);
#pragma unroll
                        for (int kk = 0; kk < UT / 16; ++kk)
                            mma_f16_ts(tmem + TM_O + 128u * t, tmem + TM_S + 128u * t + 8u * kk, sdesc_add(dv, kk * 2048),
                                       id_o, (!first || kk > 0) ? 1u : 0u);
                        if (t + 1 == ntc) mma_commit(bar(B_CVFREE + (2 * k + 1) % NCV));
                        if (last) mma_commit(bar(B_O + t));
                    }
                    if (t < ntn) {
                        scores(t, k + 1, fresh);
                        if (ok && t + 1 == ntn) mma_commit(bar(B_CVFREE + (2 * k + 2) % NCV));
                    }
                }
                c = n;
            }
            if (s_abort && issued) {   // let this thread's products land before the TMEM goes away
                mma_commit(bar(B_DRAIN));
                mbar_wait(bar(B_DRAIN), 0u, kCleanupLimitNs);
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ================================================================ widening
        Cur c;
        c.start(a, s_place);
        const int ct = tid - 128;
        constexpr int CPT = D / 16;          // 16-byte chunks of a token
        int x = 0;
        bool ok = true;
#pragma unroll 1
        for (int k = 0; k < units && ok; ++k) {
#pragma unroll 1
            for (int w = 0; w < 2; ++w, ++x) {
                const int rs = x % NRAW, cs = x % NCV;
                ok = warp_wait(B_RAWFULL + rs, (uint32_t)(x / NRAW));
                if (ok && x >= NCV) ok = warp_wait(B_CVFREE + cs, (uint32_t)(x / NCV - 1));
                if (ok && w == 1) ok = warp_wait(B_SC + k % NSC, (uint32_t)(k / NSC));
                if (!ok) break;
                const uint32_t src = sb + OFF_RAW<D> + (uint32_t)rs * RAW<D>;
                const uint32_t dst = sb + OFF_CV<D> + (uint32_t)cs * CV<D>;
                const int left = c.r.kv - c.t * UT;      // cached keys from the unit's first on
#pragma unroll 2
                for (int i = ct; i < UT * CPT; i += 128) {
                    const int row = i / CPT, ch = i % CPT;
                    uint4 u;
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                                 : "r"(src + (uint32_t)i * 16));
                    // value codes of places without a cached token: zero, so that no stale NaN
                    // meets a zero weight (stale keys only reach scores that are masked)
                    if (w == 1 && (row >= left || s_sc[(k % NSC) * 8 + (row >> 4)].y < 0.f)) u = make_uint4(0, 0, 0, 0);
                    uint32_t h[8];
                    const uint32_t cw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = decode2_h<KV>(cw[e] & 0xffffu);
                        h[2 * e + 1] = decode2_h<KV>(cw[e] >> 16);
                    }
                    // chunks 2 ch and 2 ch + 1 of the row; the second slab's lanes store the odd
                    // one first, so that a quarter warp's stores fall on distinct banks
                    const uint32_t base = dst + (uint32_t)(ch >> 2) * SLAB + (uint32_t)row * 128u;
                    const uint32_t sw = (uint32_t)(ch >> 2);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t o = (uint32_t)e ^ sw;
                        const uint32_t addr = base + ((((uint32_t)(ch & 3) * 2 + o) ^ (uint32_t)(row & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(o ? h[4] : h[0]),
                                     "r"(o ? h[5] : h[1]), "r"(o ? h[6] : h[2]), "r"(o ? h[7] : h[3])
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(B_RAWFREE + rs));
                    mbar_arrive(bar(B_CVFULL + cs));
                }
            }
            c.next_unit(a);
        }
    } else if (warp >= 8) {
        // ================================================================ softmax of tile t
        const int t = (warp - 8) >> 2, qd = warp & 3;
        const int row = 32 * qd + lane;                 // of the tile
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
        const uint32_t ts = tl + TM_S + 128u * t, to = tl + TM_O + 128u * t;
        Cur c;
        c.start(a, s_place);
        bool ok = true;
        uint32_t ns = 0, no = 0;      // units and items of this tile so far
        int k = 0;                    // unit of the CTA
#pragma unroll 1
        while (k < units && ok) {
            const int mine = min(c.nt - c.t, units - k);      // the CTA's units of this item
            const int rows = min(RB, c.r.n * a.G - c.b * RB);
            const bool first = c.t == 0, last = c.t + mine == c.nt;
            if (t == 0 && tid == 256) {
                // the CTA's entry: an item that begins here and ends elsewhere (its last)
                if (first && !last)
                    a.entry[blockIdx.x] = make_int4(cta_of(u0 + k + c.nt - 1, s_place.total, s_place.ctas), c.s, c.h, c.b);
                else if (k + mine == units)
                    a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
            }
            if (t < (rows > TR ? 2 : 1)) {
                const int lr = t * TR + row, at = c.b * RB + lr;
                const bool live = lr < rows;
                const int qi = live ? at / a.G : 0;
                const int64_t qrow = c.r.q0 + qi, hq = c.h * a.G + (at - qi * a.G);
                // ---- the row's query, normalised, to shared memory
                float cs;
                {
                    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + qrow * a.q_stride + hq * D;
                    uint4 u[D / 8];
                    float amax = 0.f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        u[i] = live ? reinterpret_cast<const uint4 *>(q)[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                                     fabsf(__uint_as_float(w[e] & 0xffff0000u))));
                    }
                    const float fac = row_factor(amax) * a.sign;
                    cs = a.scale_log2 * fabsf(1.f / fac);
                    uint8_t *dst = sm + OFF_Q<D> + (uint32_t)t * NSL * SLAB + (uint32_t)row * 128u;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = pack_h2(__uint_as_float(w[e] << 16) * fac, __uint_as_float(w[e] & 0xffff0000u) * fac);
                        *reinterpret_cast<uint4 *>(dst + (i >> 3) * SLAB + (((uint32_t)(i & 7) ^ (uint32_t)(row & 7)) << 4)) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_Q + t));
                }
                const int lim = live ? seen_by(c.r, qi) : 0;
                float M = -INFINITY, l = 0.f;
#pragma unroll 1
                for (int j = 0; j < mine && ok; ++j) {
                    const int kk = k + j, sc = (kk % NSC) * 8, tok0 = (c.t + j) * UT;
                    // the scores first: a tile that sat out items is then at this unit, and the
                    // scale slot's phase is the one before or after its publication
                    ok = warp_wait(B_S + t, ns++) && warp_wait(B_SC + kk % NSC, (uint32_t)(kk / NSC));
                    if (!ok) break;
                    tc_fence_after();
                    // which of the unit's keys this row sees; all of them in most units
                    bool part = tok0 + UT > lim;
#pragma unroll
                    for (int i = 0; i < 8; ++i) part |= s_sc[sc + i].y < 0.f;
                    part = __any_sync(0xffffffffu, part);
                    // pass 1: the row's maximum
                    float mx = -INFINITY;
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        float v[32];
                        tmem_ld32(ts + 32u * cb, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 s4 = s_sc[sc + 2 * cb + i];
                            float m = -INFINITY;
                            if (part) {
                                const int see = s4.y < 0.f ? 0 : lim - (tok0 + 32 * cb + 16 * i);
#pragma unroll
                                for (int e = 0; e < 16; ++e) m = fmaxf(m, e < see ? v[16 * i + e] : -INFINITY);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; ++e) m = fmaxf(m, v[16 * i + e]);
                            }
                            if (m != -INFINITY) mx = fmaxf(mx, fmaf(m, cs * s4.x, s4.z));
                        }
                    }
                    if (__any_sync(0xffffffffu, mx > M + kv8::kTau)) {
                        const float m = fmaxf(M, ceilf(mx)), w = part_weight(M, m);
                        M = m;
                        l *= w;
                        if (j > 0) {      // the sums of the units before (their products have landed)
#pragma unroll 1
                            for (int cb = 0; cb < D / 32; ++cb) {
                                float o[32];
                                tmem_ld32(to + 32u * cb, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= w;
                                tmem_st32(to + 32u * cb, o);
                            }
                        }
                    }
                    // pass 2: the weights, over the scores
                    const float ref = kv8::kOff - (M == -INFINITY ? 0.f : M);
#pragma unroll
                    for (int cb = 0; cb < 4; ++cb) {
                        float v[32];
                        uint32_t p[16];
                        tmem_ld32(ts + 32u * cb, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 s4 = s_sc[sc + 2 * cb + i];
                            const float kf = cs * s4.x, add = s4.z + ref;
                            const int see = !part ? 16 : s4.y < 0.f ? 0 : lim - (tok0 + 32 * cb + 16 * i);
                            float sum = 0.f;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float p0 = ex2(fmaf(v[16 * i + e], kf, add));
                                float p1 = ex2(fmaf(v[16 * i + e + 1], kf, add));
                                if (part) {
                                    p0 = e < see ? p0 : 0.f;
                                    p1 = e + 1 < see ? p1 : 0.f;
                                }
                                sum += p0 + p1;
                                p[8 * i + (e >> 1)] = pack_h2(p0, p1);
                            }
                            l = fmaf(sum, s4.w, l);
                        }
                        tmem_st16(ts + 16u * cb, p);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P + t));
                }
                // ---- the item's sums
                if (ok) ok = warp_wait(B_O + t, no++);
                if (ok) {
                    tc_fence_after();
                    const bool whole = first && last;
                    const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                    const int64_t slot = ((int64_t)blockIdx.x * 2 + (first ? 1 : 0)) * RB + lr;
                    const int64_t orow = qrow * a.Hq + hq;
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        float o[32];
                        tmem_ld32(to + 32u * cb, o);
                        tmem_wait_ld();
                        if (!live) continue;
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= inv;
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + orow * D + 32 * cb;
#pragma unroll
                            for (int e = 0; e < 32; e += 8) Vec16<__nv_bfloat16>::store(dst + e, o + e);
                        } else {
                            float *dst = a.part_o + slot * D + 32 * cb;
#pragma unroll
                            for (int e = 0; e < 32; e += 4) Vec16<float>::store(dst + e, o + e);
                        }
                    }
                    if (live && whole && a.lse)
                        a.lse[orow] = l == 0.f ? -INFINITY
                                               : ((M == -INFINITY ? 0.f : M) - kv8::kOff + log2f(l)) * 0.693147180559945f;
                    if (live && !whole) *reinterpret_cast<float2 *>(a.part_ml + 2 * slot) = make_float2(M, l);
                    tc_fence_before();
                }
            }
            k += mine;
            c.next_of_item(a);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (s_abort && tid == 0) a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (warp == 1) tmem_dealloc(tmem, TM_COLS);
    grid_launch_dependents();
}

template <Kv8 KV, int D>
cudaError_t launch_tile_d(const AttnArgs &a, int ctas, int rows, cudaStream_t s) {
    auto kernel = kv8_tile_kernel<KV, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tl::SMEM<D>);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)ctas, tl::NT, tl::SMEM<D>, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_merge<__nv_bfloat16, D, tl::RB, 1>(a, ctas, rows, s);
}

}  // namespace

cudaError_t launch_kv8_tile(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                            const float *k_scale, const float *v_scale, const int *table,
                            const int *kv_len, const int *cu_q, float scale, void *out, float *lse, int S,
                            int max_q, int total_q, int Hq, int Hkv, int D, int W, int page, int N, Kv8 kv,
                            void *ws, cudaStream_t s) {
    const int ctas = sm_count();
    AttnArgs a{};
    a.q = q, a.q_stride = q_stride, a.kc = static_cast<const uint8_t *>(k_cache);
    a.vc = static_cast<const uint8_t *>(v_cache);
    a.ks = k_scale, a.vs = v_scale, a.table = table, a.kv_len = kv_len;
    a.cu_q = cu_q, a.scale_log2 = fabsf(scale) * 1.4426950408889634f, a.sign = scale < 0.f ? -1.f : 1.f;
    a.out = out, a.lse = lse;
    place_parts(a, ws, ctas, tl::RB);
    a.S = S, a.total_q = total_q, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.W = W, a.N = N;
    a.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    a.limit_ns = wait_limit_ns();
    const int64_t rows64 = (int64_t)max_q * a.G;
    const int rows = rows64 > tl::RB ? tl::RB : (int)rows64;
    if (D == 128)
        return kv == Kv8::E4M3 ? launch_tile_d<Kv8::E4M3, 128>(a, ctas, rows, s)
                               : launch_tile_d<Kv8::INT8, 128>(a, ctas, rows, s);
    return kv == Kv8::E4M3 ? launch_tile_d<Kv8::E4M3, 64>(a, ctas, rows, s)
                           : launch_tile_d<Kv8::INT8, 64>(a, ctas, rows, s);
}

cudaError_t take_kv8_tile_error_word(unsigned *value) { return take_error_word(value); }

}  // namespace gdr
