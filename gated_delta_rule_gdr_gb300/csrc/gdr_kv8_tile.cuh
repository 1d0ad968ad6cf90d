// gdr_kv8_tile.cuh -- attention over the 8-bit paged cache for more than 16 bf16 query rows a
// cached head: prompts, chunks of prompts against a long cache, drafted tokens, the queries of requests
// that share a prefix (gdr_kv8_attn, gdr_kv8_attn_shared).
//
// The same mathematics as the split kernel's (gdr_kv8_split.cuh): with a whole-number reference
// exponent M for each row over x_j + log2 vs,
//   P_j = 2^(x_j + log2 vs - M + 14),  O += P_j vcode_j,  l += P_j / vs,  o = O / l.
//
// A unit is 128 keys; an item's rows (row = query x group of heads) are tiles of 128.  A tile's
// scores S (128 x 128 fp32) and sums O live in TMEM; its weights go back over S as halves and
// are the A operand of the second product from there, so that they never touch shared memory.
// The codes come by bulk copies (a page's block of a head is contiguous) and are widened to
// halves in the tensor core's swizzled layout: keys K-major, values MN-major from the same
// [token][64 values] rows, so values need no transpose.
//
// Three forms, by the most rows of a cached head that a request has:
//   PAIR (above 128): items of 256 rows.  Two tiles of different rows share every key, the
//       softmax of one runs under the products of the other.
//   one tile (65 to 128): its units alternate between the two score and sum buffers.
//   copies (up to 64 or 32, NC = 2 or 4): the tile holds the rows NC times, and a copy's warps
//       take the softmax of their half or quarter of the unit's keys only, with weights of zero
//       elsewhere: what a warp does a unit is 1 / NC, and all four parts of the SM work at the
//       exponentials.  The copies' sums are joined at the item's end.
//
// Bounds.  PAIR: the two products, 4 rows keys D flops.  Measured: 1000 tokens of 4 heads a
// cached head, 8 of those, on 65 k keys (1.07 TFLOP) 0.982 ms = 1.09 PFLOP/s, 56 % of a large
// matrix product's measured rate; four prompts of 4096 (275 GFLOP counting only what is seen)
// 0.343 ms.  The tensor cores wait for the softmax's chain of TMEM loads, maxima, exponentials
// and stores (two tiles hide about half of it).
// Copies: the cache's bytes.  32 requests of 5 x 8 rows on up to 32 k keys (555 MB) 0.156 ms =
// 3.6 TB/s.  Of the 2400 cycles that a unit takes the widening warps work 1500 and wait 700 for a
// slot that the products give back; shared memory is busy for as much: a unit's 32 KB of codes
// are read once, written widened (64 KB) and read by the products with the queries (96 KB).
//
// Warps: 0 and 3 load (keys; values and scales), 1 and 2 issue the products (1 owns the TMEM),
// 4-5 widen keys, 6-7 values, 8-11 and 12-15 the softmax of buffer 0 and 1, a thread a row:
// maxima and sums never leave the thread.  No barrier spans the CTA inside the loop; every
// wait is bounded.

#pragma once

#include "gdr_kv8_attn.cuh"

#include <cmath>

namespace gdr {
namespace {

namespace tl {
constexpr int NT = 512;
constexpr int TR = 128, UT = 128;                // rows of a tile, keys of a unit
constexpr int NRAW = 4, NSC = 4;                 // raw slots (keys and values in turn), scale slots
constexpr uint32_t SLAB = 128 * 128;             // 128 rows x 64 halves
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;   // buffer b at + 128 b
constexpr int MAXCV = 4;
enum : int {
    B_RAWFULL = 0, B_RAWFREE = B_RAWFULL + NRAW, B_CVFULL = B_RAWFREE + NRAW, B_CVFREE = B_CVFULL + MAXCV,
    B_SC = B_CVFREE + MAXCV, B_Q = B_SC + NSC, B_S = B_Q + 2, B_PU = B_S + 2, B_P = B_PU + 2, B_O = B_P + 2,
    B_ML = B_O + 2, B_OFREE = B_ML + 1, B_DRAIN = B_OFREE + 1, B_U = B_DRAIN + 2,
    B_X = B_U + 2, NUM_BARS = B_X + 1
};
template <int D, bool PAIR, int NC> struct Lay {
    static constexpr int RB = PAIR ? kKv8TileRows : TR / NC;   // rows of an item
    // What an item's ends cost, in units.  PAIR 0 / 2 / 3 / 4: four prompts of 4096 0.415 / 0.352 /
    // 0.347 / 0.347 ms; else 0 / 6 / 8 / 12: 200 requests of 5 x 8 rows on up to 2000 keys 0.178 /
    // 0.120 / 0.120 / 0.125, 32 on up to 32 k 0.187 / 0.158 / 0.155 / 0.159.
    static constexpr int ITEM = PAIR ? 3 : 8;
    static constexpr uint32_t XR = (TR - TR / NC) * 128;  // sums of the copies that are joined, 32 columns (NC > 1)
    static constexpr int NCV = PAIR ? 3 : 4;              // widened slots
    static constexpr uint32_t RAW = UT * D, CV = UT * D * 2;
    static constexpr uint32_t OFF_Q = 0;                  // one tile, or two
    static constexpr uint32_t QT = (PAIR ? 2 : 1) * TR * D * 2;
    static constexpr uint32_t OFF_CV = QT > 2 * XR ? QT : 2 * XR;
    static constexpr uint32_t OFF_RAW = OFF_CV + NCV * CV;
    static constexpr uint32_t OFF_SC = OFF_RAW + NRAW * RAW;     // [NSC][8 groups]{ks, vs, log2 vs, 1/vs}
    static constexpr uint32_t OFF_ML = OFF_SC + NSC * 8 * 16;    // [TR]{M, l} of buffer 1 (not PAIR)
    static constexpr uint32_t SMEM = OFF_ML + (PAIR ? 0 : TR * 8);   // 1024-byte aligned by its declaration
    static_assert(SMEM + 1024 <= 232448, "exceeds 227 KB of shared memory per CTA");
};
}  // namespace tl

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One lane of a converged warp (always the same one).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A warp's wait for up to 32 barriers at once, a lane's own each (need: this lane has one):
// a barrier is a trip to shared memory, which the products keep busy, and one trip serves
// them all.  Bounded as role_wait; true once every lane's phase has completed.
__device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, bool need, uint64_t limit_ns,
                                            volatile int *abort) {
    const uint64_t t0 = global_timer_ns();
    bool give_up = limit_ns == 0;
    while (true) {
        if (!give_up) {
            const bool done = !need || mbar_try_wait_hint(bar, parity, kWaitSliceNs);
            if (__all_sync(0xffffffffu, done)) return true;
            if (*abort) give_up = true;
            if (global_timer_ns() - t0 > limit_ns) give_up = true;
        }
        if (__any_sync(0xffffffffu, give_up)) {
            if (give_up && !*abort) {
                *abort = 1;
                atomicOr(&g_device_error_word, kDevErrTimeout);
            }
            __syncwarp();
            return false;
        }
    }
}
__device__ __forceinline__ bool warp_wait_all(uint32_t bar, uint32_t parity, bool need, uint64_t limit_ns,
                                              volatile int *abort) {
    const bool done = !need || mbar_test_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    return warp_wait_slow(bar, parity, need, limit_ns, abort);
}

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

// A query row of the item that block b of RB rows is.
__device__ __forceinline__ void note_prefix(TileRow &, const Request &) {}
__device__ __forceinline__ void note_prefix(SharedRow &t, const SharedRequest &r) { t.pre = r.skip > 0; }
template <int RB, class A>
__device__ __forceinline__ typename A::Row tile_row(const A &a, const Cursor<RB, tl::UT, A> &c, int lr) {
    typename A::Row t;
    note_prefix(t, c.r);
    const int at = c.b * RB + lr;
    t.live = lr < RB && at < c.r.n * a.G;
    const int i = t.live ? at / a.G : 0;
    t.qrow = c.r.q0 + i;
    t.hq = c.h * a.G + (t.live ? at - i * a.G : 0);
    t.lim = t.live ? seen_by(a, c.r, i) : 0x3fffffff;   // a row that is not there needs no mask
    return t;
}

// The queries of a warp's 32 rows (rows row0 .. row0 + 31 of the item at c), in two steps:
// begin_queries starts their copies, raw, to the K-major tile's rows 32 qd on (D / 8 lanes a
// row: a lane reading its own row would touch 32 lines an instruction); end_queries, in the
// same lanes' pieces, turns them to halves and returns the rows' score factor.  All 32 rows are
// scaled by one power of two that brings the largest magnitude below 2^15, if every piece of 8
// values reaches 2^-14 of it (the smallest row then keeps values good to 2^-25 of its own
// largest); else each row by one of its own, so that a row depends on no other (a common factor
// loses a row beside one 2^28 times larger).  Rows apart are marked by the factor's sign, and
// their scores are brought back where masks are applied, off the usual way: a factor of its own
// for every row and item took 0.376 ms against 0.350 for four prompts of 4096, 1.044 against
// 0.994 for the chunk on 65 k.  Loops, not unrolled code: they run once an item, from cold caches.
template <int D>
__device__ __forceinline__ uint32_t query_place(int qd, int i) {    // of this lane's piece of step i
    constexpr int LPR = D / 8, RPI = 32 / LPR;    // lanes a row, rows a step
    const uint32_t lane = threadIdx.x & 31, piece = lane % LPR, row = 32u * qd + RPI * i + lane / LPR;
    return (piece >> 3) * tl::SLAB + row * 128u + (((piece & 7u) ^ (row & 7u)) << 4);
}
template <int D, int RB, class A>
__device__ __forceinline__ void begin_queries(const A &a, const Cursor<RB, tl::UT, A> &c, int row0, int qd, uint32_t dst) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, IT = 32 / RPI;
    const int lane = threadIdx.x & 31;
    const int rows = min(RB, c.r.n * a.G - c.b * RB), first = row0 + lane / LPR;
    int tok = (c.b * RB + first) / a.G, g = c.b * RB + first - tok * a.G;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)c.h * a.G * D + (lane % LPR) * 8;
#pragma unroll 1
    for (int i = 0; i < IT; ++i) {
        const bool live = first + RPI * i < rows;
        const void *src = live ? q + (int64_t)(c.r.q0 + tok) * a.q_stride + (int64_t)g * D : q;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + query_place<D>(qd, i)), "l"(src),
                     "r"(live ? 16 : 0)      // a row that is not there: zeros
                     : "memory");
        for (g += RPI; g >= a.G; g -= a.G) ++tok;
    }
}
__device__ __forceinline__ uint32_t piece_magnitude(const uint4 &u) {     // patterns compare as magnitudes do
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(m & 0xffff0000u, m << 16);
}
__device__ __forceinline__ uint4 piece_to_halves(const uint4 &u, float fac) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        h[e] = pack_h2(__uint_as_float(w[e] << 16) * fac, __uint_as_float(w[e] & 0xffff0000u) * fac);
    return make_uint4(h[0], h[1], h[2], h[3]);
}
// The pattern of 1 / |fac|, a power of two.
__device__ __forceinline__ uint32_t inverse(float fac) { return 0x7f000000u - (__float_as_uint(fac) & 0x7fffffffu); }
// A factor for each row; its inverse's exponent is left in s_fac, at the row's softmax thread.
// (Inlined, it changes the softmax loop's registers: 1.035 ms against 0.994 for the chunk on 65 k.)
__device__ __forceinline__ uint8_t *fac_of(uint8_t *s_fac) { return s_fac + (threadIdx.x & (2 * tl::TR - 1)); }
template <int D>
__device__ __noinline__ void rows_apart(int qd, uint8_t *dst, float sign, uint8_t *s_fac) {
    constexpr int LPR = D / 8, RPI = 32 / LPR, IT = 32 / RPI;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int i = 0; i < IT; ++i) {
        uint4 *p = reinterpret_cast<uint4 *>(dst + query_place<D>(qd, i));
        const uint4 u = *p;
        uint32_t m = piece_magnitude(u);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float fac = row_factor(__uint_as_float(m)), own = __shfl_sync(0xffffffffu, fac, lane % RPI * LPR);
        if (lane / RPI == i) *fac_of(s_fac) = (uint8_t)(inverse(own) >> 23);
        *p = piece_to_halves(u, fac * sign);
    }
}
template <int D>
__device__ __forceinline__ float end_queries(const AttnArgs &a, int qd, uint8_t *dst, uint8_t *s_fac) {
    constexpr int IT = D / 8;
    asm volatile("cp.async.wait_all;" ::: "memory");
    uint32_t m = 0, least = ~0u;          // of the pieces, those of zeros aside
#pragma unroll 4
    for (int i = 0; i < IT; ++i) {
        const uint32_t x = piece_magnitude(*reinterpret_cast<const uint4 *>(dst + query_place<D>(qd, i)));
        m = max(m, x);
        least = min(least, x - 1u);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    least = __reduce_min_sync(0xffffffffu, least);
    if (m >= 0x7f800000u || least + (14u << 23) < m) {
        rows_apart<D>(qd, dst, a.sign, s_fac);
        return -a.scale_log2;
    }
    const float fac = row_factor(__uint_as_float(m)) * a.sign;
#pragma unroll 2
    for (int i = 0; i < IT; ++i) {
        uint4 *p = reinterpret_cast<uint4 *>(dst + query_place<D>(qd, i));
        *p = piece_to_halves(*p, fac);
    }
    return a.scale_log2 * __uint_as_float(inverse(fac));
}

// One unit of one row, the upper half's keys (64 on) first: scores from TMEM, M moved on where a
// score exceeds it by much, the weights as halves to the upper columns (kP on; they go over
// scores that have been read by then), l.  By halves, or in a loop over chunks of 32 keys
// whose scores are read twice: the chunked code is a quarter of the size, and where many
// warps with little to do share the instruction caches their misses were the largest stall
// (3.7 of 10 warps waiting for instructions).
// GR: groups of a half (64 keys) with a scale of their own: one where pages hold 64 tokens or
// more, else four.
constexpr uint32_t kP = 64;
template <int GR> struct RowUnit {
    const float4 *sc;              // the unit's scales: {ks, vs, log2 vs, 1 / vs} a group of 16
    int see;                       // keys of the unit that the row sees
    bool part;                     // some row of the warp sees fewer than all, a page is gone, or rows are apart
    float cs;                      // negative: rows apart
    uint8_t *fac;
    float4 held[2];                // GR 1: the scales of the two halves (PAIR; NC 2: of the warp's, twice)
    __device__ __forceinline__ float4 scales(int h, int i) const { return GR == 1 ? (h ? held[1] : held[0]) : sc[4 * h + i]; }
};
// A factor of at least 2^-126 keeps masked scores at -inf where a scale is zero.
__device__ __forceinline__ float unit_factor(float cs, float ks) { return fmaxf(fabsf(cs) * ks, 1.2e-38f); }
template <int GR, int N>
__device__ __forceinline__ void bring_back(const RowUnit<GR> &u, float (&v)[N]) {
    if (__float_as_int(u.cs) >= 0) return;
    const float k = __uint_as_float((uint32_t)*fac_of(u.fac) << 23);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] *= k;
}
template <int GR>
__device__ __forceinline__ void load_chunk(uint32_t ts, int ch, const RowUnit<GR> &u, float (&v)[32]) {
    tmem_ld32(ts + 32u * ch, v);
    tmem_wait_ld();
    if (u.part) {
        bring_back(u, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = u.sc[2 * ch + i].y < 0.f ? 0 : u.see - 32 * ch - 16 * i;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e >= n) v[16 * i + e] = -INFINITY;
        }
    }
}
// The largest exponent of some keys, and the largest of those that are not in its group (16 keys,
// or a half of what is looked at where one scale covers it).
struct Largest {
    float mx = -INFINITY, next = -INFINITY;
    __device__ __forceinline__ void add(float x) {
        next = fmaxf(next, fminf(mx, x));
        mx = fmaxf(mx, x);
    }
};
template <int N, typename X>
__device__ __forceinline__ float max_of(X x) {
    float m = fmaxf(x(0), x(1));
#pragma unroll
    for (int e = 2; e < N; e += 2) m = fmaxf(fmaxf(m, x(e)), x(e + 1));
    return m;
}
template <int GR>
__device__ __forceinline__ void chunk_max(const float (&v)[32], int ch, const RowUnit<GR> &u, Largest &r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 s4 = u.sc[GR == 1 ? 4 * (ch >> 1) : 2 * ch + i];
        r.add(fmaf(max_of<16>([&](int e) { return v[16 * i + e]; }), unit_factor(u.cs, s4.x), s4.z));
    }
}
template <int GR>
__device__ __forceinline__ float chunk_weights(uint32_t ts, int ch, const RowUnit<GR> &u, const float (&v)[32], float ref, float l) {
    constexpr int N = GR == 1 ? 32 : 16;
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 32 / N; ++i) {
        const float4 s4 = u.sc[GR == 1 ? 4 * (ch >> 1) : 2 * ch + i];
        const float kf = unit_factor(u.cs, s4.x), add = s4.z + ref;
        const uint64_t kf2 = f2_pack(kf, kf), add2 = f2_pack(add, add);
        uint64_t sum = 0;
#pragma unroll
        for (int e = N * i; e < N * i + N; e += 2) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(v[e], v[e + 1]), kf2, add2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum = f2_add(sum, f2_pack(p0, p1));
            p[e >> 1] = pack_h2(p0, p1);
        }
        float s0, s1;
        f2_unpack(sum, s0, s1);
        l = fmaf(s0 + s1, s4.w, l);
    }
    tmem_st16(ts + kP + 16u * ch, p);
    return l;
}
// By halves: 64 scores in registers, read once.
template <int GR>
__device__ __forceinline__ void load_half(uint32_t ts, int h, const RowUnit<GR> &u, float (&v)[2][32]) {
    tmem_ld32(ts + 64u * h, v[0]);
    tmem_ld32(ts + 64u * h + 32u, v[1]);
    tmem_wait_ld();
    if (u.part) {
        bring_back(u, v[0]);
        bring_back(u, v[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = u.sc[4 * h + i].y < 0.f ? 0 : u.see - 64 * h - 16 * i;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e >= n) v[i >> 1][16 * (i & 1) + e] = -INFINITY;
        }
    }
}
template <int GR>
__device__ __forceinline__ Largest half_max(const float (&v)[2][32], int h, const RowUnit<GR> &u) {
    Largest r;
#pragma unroll
    for (int i = 0; i < (GR == 1 ? 2 : 4); ++i) {
        constexpr int N = GR == 1 ? 32 : 16;
        const float4 s4 = u.scales(h, i);
        r.add(fmaf(max_of<N>([&](int e) { return v[(N * i + e) >> 5][(N * i + e) & 31]; }), unit_factor(u.cs, s4.x), s4.z));
    }
    return r;
}
template <int GR>
__device__ __forceinline__ float half_weights(uint32_t ts, int h, const RowUnit<GR> &u, const float (&v)[2][32], float ref,
                                              float l) {
    constexpr int N = 64 / GR;
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
        uint32_t p[16];
        uint64_t kf2 = 0, add2 = 0, sum = 0;
        float iv = 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            if (e % N == 0) {
                const float4 s4 = u.scales(h, (32 * cb + e) / 16);
                const float kf = unit_factor(u.cs, s4.x), add = s4.z + ref;
                kf2 = f2_pack(kf, kf), add2 = f2_pack(add, add);
                iv = s4.w;
                sum = 0;
            }
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(v[cb][e], v[cb][e + 1]), kf2, add2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum = f2_add(sum, f2_pack(p0, p1));
            p[e >> 1] = pack_h2(p0, p1);
            if ((e + 2) % N == 0 || e == 30) {
                float s0, s1;
                f2_unpack(sum, s0, s1);
                l = fmaf(s0 + s1, iv, l);
            }
        }
        tmem_st16(ts + kP + 32u * h + 16u * cb, p);
    }
    return l;
}
// Moves M to hold scores whose largest exponent is mx, and the sums so far with it.  That is a trip
// through the TMEM, so M is set kRoom above the largest score and holds what exceeds that by up to
// 8.5: rare (3.5, 2.5 or 1.5: four prompts of 4096 0.406, 0.424, 0.438 ms against 0.343, the chunk on
// 65 k 1.06, 1.09, 1.12 against 0.985).  But the room is lost to the small weights, and they are
// all of the output where the largest one's value is nothing.  So a row whose largest score stands
// 16 (2^16 in weight) above the scores before it goes without; its first ones are compared with
// `next`, the largest of the keys that are not beside it, or (`lower`) with the half that comes
// second.
// settled() waits until no product writes the sums.
constexpr float kRoom = 7.f, kAlone = 16.f;
template <int D, typename Settled>
__device__ __forceinline__ bool move_reference(uint32_t to, float mx, float next, bool rescale, bool lower, float &M, float &l,
                                               Settled settled) {
    const bool alone = lower && mx < M - (kRoom + kAlone) && mx > -INFINITY;
    if (!__any_sync(0xffffffffu, mx > M + kv8::kTau || alone)) return true;
    float m = fmaxf(M, ceilf(mx) + kRoom);
    if (alone || mx > (M == -INFINITY ? next : M - kRoom) + kAlone) m -= kRoom;
    const float w = part_weight(M, m);
    M = m;
    l *= w;
    if (!rescale) return true;
    if (!settled()) return false;
#pragma unroll 1
    for (int cb = 0; cb < D / 8; ++cb) {
        uint32_t o[8];
        tmem_ld8(to + 8u * cb, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w);
        tmem_st8(to + 8u * cb, o);
    }
    tmem_wait_st();
    return true;
}
// publish(h): called when the weights of half h (1, then 0) are in place; upper_done(): waits
// for the products of the upper half (false from either: give up).  BY_HALVES (the tensor
// cores bound): a half's scores stay in registers between the maximum and the weights; the
// lower half's maximum is taken after the upper half's weights are out, and waits for their
// products if it moves M.  Else (the cache's bytes bound): chunk by chunk, all maxima first, and
// nothing here waits for a product: with one warp issuing for both buffers, in order, such a
// wait could meet one for the next item's queries, which in turn wait for this unit.  Chunks
// measured against halves: 0.274 / 0.352 ms for 32 requests of 5 x 8 rows on up to 32 k keys in
// one tile, 1.48 / 1.16 ms for pairs at 1000 tokens on 65 k.  NC > 1: the keys of this warp's
// copy alone, in registers (one tile against two copies 0.225 / 0.219 ms there).
template <int D, int GR, bool BY_HALVES, int NC, typename Publish, typename UpperDone>
__device__ __forceinline__ bool softmax_unit(uint32_t ts, uint32_t to, const RowUnit<GR> &u, int copy, bool rescale, float &M, float &l,
                                             Publish publish, UpperDone upper_done) {
    auto ref = [&]() { return kv8::kOff - (M == -INFINITY ? 0.f : M); };
    if constexpr (BY_HALVES) {
        float v[2][32];
        load_half<GR>(ts, 1, u, v);
        // the earlier units' products have landed: the scores' barrier came after them
        const float mx = half_max<GR>(v, 1, u).mx;
        move_reference<D>(to, mx, mx, rescale, false, M, l, []() { return true; });
        l = half_weights<GR>(ts, 1, u, v, ref(), l);
        tmem_wait_st();
        if (!publish(1)) return false;
        load_half<GR>(ts, 0, u, v);
        if (!move_reference<D>(to, half_max<GR>(v, 0, u).mx, -INFINITY, true, !rescale, M, l, upper_done)) return false;
        l = half_weights<GR>(ts, 0, u, v, ref(), l);
        tmem_wait_st();
        return publish(0);
    } else if constexpr (NC > 1) {
        // the copy's keys only, from registers; the other copies' weigh nothing in its rows
        if constexpr (NC == 2) {
            float v[2][32];
            load_half<GR>(ts, copy, u, v);
            const Largest x = half_max<GR>(v, copy, u);
            move_reference<D>(to, x.mx, rescale ? x.mx : x.next, rescale, false, M, l, []() { return true; });
            l = half_weights<GR>(ts, copy, u, v, ref(), l);
        } else {
            float v[32];
            load_chunk<GR>(ts, copy, u, v);
            Largest x;
            chunk_max<GR>(v, copy, u, x);
            move_reference<D>(to, x.mx, rescale ? x.mx : x.next, rescale, false, M, l, []() { return true; });
            l = chunk_weights<GR>(ts, copy, u, v, ref(), l);
        }
        const uint32_t zero[16] = {};
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch)
            if (ch / (4 / NC) != copy) tmem_st16(ts + kP + 16u * ch, zero);
        tmem_wait_st();
        return publish(1) && publish(0);
    } else {
        float v[32];
        Largest x;
#pragma unroll 1
        for (int ch = 3; ch >= 0; --ch) {
            load_chunk<GR>(ts, ch, u, v);
            chunk_max<GR>(v, ch, u, x);
        }
        move_reference<D>(to, x.mx, rescale ? x.mx : x.next, rescale, false, M, l, []() { return true; });
#pragma unroll 1
        for (int ch = 3; ch >= 0; --ch) {
            load_chunk<GR>(ts, ch, u, v);
            l = chunk_weights<GR>(ts, ch, u, v, ref(), l);
            if (ch & 1) continue;
            tmem_wait_st();
            if (!publish(ch >> 1)) return false;
        }
        return true;
    }
}

// A row's result: the output, or the part that the merge kernel joins.  A lane writes its own
// row: 32 bytes a store where everything is so aligned, whole sectors.
__device__ __forceinline__ void store32(void *p, const uint32_t *w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// How a row ends: what its sums are multiplied with, and in the second pass over a shared prefix also the
// first one's sums with their factor.
struct RowEnd {
    float f;
};
struct SharedEnd {
    float f, fx;
    const float *pre;        // null: there are none
};
template <int D>
__device__ __forceinline__ RowEnd end_row(const AttnArgs &, const TileRow &, bool, float, float &l) {
    return RowEnd{l == 0.f ? 0.f : 1.f / l};
}
template <int D>
__device__ __forceinline__ RowEnd end_row(const SharedArgs<true> &, const TileRow &, bool, float, float &) { return RowEnd{1.f}; }
template <int D>
__device__ __forceinline__ SharedEnd end_row(const SharedArgs<false> &a, const SharedRow &t, bool whole, float &M, float &l) {
    SharedEnd x{1.f, 0.f, nullptr};
    if (whole && t.live && t.pre) {
        const int64_t row = (int64_t)t.qrow * a.Hq + t.hq;
        const float2 m = a.pre_ml[row];
        const float top = fmaxf(M, m.x);
        x.f = join_weight(M, top), x.fx = join_weight(m.x, top);
        x.pre = a.pre_o + row * D;
        l = fmaf(x.fx, m.y, l * x.f);
        M = top;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    x.f *= inv, x.fx *= inv;
    return x;
}
// Where a row's complete sums stay, null: they are written out.
template <int D> __device__ __forceinline__ float *left_at(const AttnArgs &, const TileRow &) { return nullptr; }
template <int D> __device__ __forceinline__ float *left_at(const SharedArgs<true> &a, const TileRow &t) {
    return a.pre_o + ((int64_t)t.qrow * a.Hq + t.hq) * D;
}
// 16 values from `at` on (a store's: the memory clobber between two keeps the second's loads behind the
// first, and registers are short here).
__device__ __forceinline__ void join_values(const RowEnd &, int, float *) {}
__device__ __forceinline__ void join_values(const SharedEnd &x, int at, float *o) {
    if (!x.pre) return;
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        const float4 p = *reinterpret_cast<const float4 *>(x.pre + at + e);
        o[e] = fmaf(x.fx, p.x, o[e]), o[e + 1] = fmaf(x.fx, p.y, o[e + 1]);
        o[e + 2] = fmaf(x.fx, p.z, o[e + 2]), o[e + 3] = fmaf(x.fx, p.w, o[e + 3]);
    }
}
template <int D, int RB, class A, class End>
__device__ __forceinline__ void write_chunk(const A &a, const typename A::Row &t, bool whole, int64_t slot, int cb,
                                            const End &end, float (&o)[32]) {
    if (!t.live) return;
    uint32_t w[32];
    float *left = left_at<D>(a, t);
    if (whole && !left) {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)t.qrow * a.Hq + t.hq) * D + 32 * cb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[16 * h + e] *= end.f;
            join_values(end, 32 * cb + 16 * h, o + 16 * h);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[16 * h + 2 * e], o[16 * h + 2 * e + 1]);
            store32(dst + 16 * h, w, a.wide);
        }
    } else {
        float *dst = (whole ? left : a.part_o + slot * D) + 32 * cb;
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) store32(dst + 8 * e, w + 8 * e, a.wide);
    }
}
__device__ __forceinline__ bool leave_stats(const AttnArgs &, int64_t, float, float) { return false; }
__device__ __forceinline__ bool leave_stats(const SharedArgs<true> &a, int64_t row, float M, float l) {
    a.pre_ml[row] = make_float2(M, l);
    return true;
}
template <class A>
__device__ __forceinline__ void write_stats(const A &a, const typename A::Row &t, bool whole, int64_t slot, float M, float l) {
    if (!t.live) return;
    const int64_t row = (int64_t)t.qrow * a.Hq + t.hq;
    if (!whole)
        *reinterpret_cast<float2 *>(a.part_ml + 2 * slot) = make_float2(M, l);
    else if (!leave_stats(a, row, M, l) && a.lse)
        a.lse[row] = l == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) - kv8::kOff + log2f(l)) * 0.693147180559945f;
}

template <Kv8 KV, int D, bool PAIR, int NC, int GR, class A>
__global__ void __launch_bounds__(tl::NT, 1) kv8_tile_kernel(const A a) {
    using namespace tl;
    using L = Lay<D, PAIR, NC>;
    constexpr int RB = L::RB, NCV = L::NCV, NSL = D / 64;
    using Cur = Cursor<RB, UT, A>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    __shared__ __align__(8) uint64_t s_bar[NUM_BARS];
    __shared__ FirstPlace<A> s_place;
    __shared__ int64_t s_scan[2 * NT / 32];
    __shared__ uint32_t s_tmem;
    __shared__ int s_gone[NSC];
    __shared__ float s_cs[4];        // one-tile form: the score factors of the tile's four groups of rows
    __shared__ uint8_t s_fac[2 * TR];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return smem_u32(&s_bar[i]); };
    float4 *s_sc = reinterpret_cast<float4 *>(sm + L::OFF_SC);
    const int P = 1 << a.page_log2;

    if (tid == 0) {
        for (int i = 0; i < NRAW; ++i) {
            mbar_init(bar(B_RAWFULL + i), 1);
            mbar_init(bar(B_RAWFREE + i), 2);
        }
        for (int i = 0; i < NCV; ++i) {
            mbar_init(bar(B_CVFULL + i), 2);
            mbar_init(bar(B_CVFREE + i), PAIR ? 2 : 1);
        }
        for (int i = 0; i < NSC; ++i) mbar_init(bar(B_SC + i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_Q + i), 4);
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_PU + i), 4);
            mbar_init(bar(B_P + i), 4);
            mbar_init(bar(B_DRAIN + i), 1);
            mbar_init(bar(B_U + i), 1);
            mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_ML), 4);
        mbar_init(bar(B_OFREE), 4);
        mbar_init(bar(B_X), 4);
        s_abort = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();
    find_place<RB, UT, NT, L::ITEM>(a, &s_place, s_scan);
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
    // one barrier (b0), or several: lane i has b_i, of phase n_i; a negative b_i is none
    auto warp_wait = [&](int b, uint32_t n) { return warp_wait_all(bar(b), n & 1u, true, a.limit_ns, &s_abort); };
    auto warp_wait3 = [&](int b0, uint32_t n0, int b1, uint32_t n1, int b2, uint32_t n2) {
        const int b = lane == 0 ? b0 : lane == 1 ? b1 : lane == 2 ? b2 : -1;
        const uint32_t n = lane == 0 ? n0 : lane == 1 ? n1 : n2;
        return warp_wait_all(bar(max(b, 0)), n & 1u, b >= 0, a.limit_ns, &s_abort);
    };
    auto tiles_of = [&](const Cur &c) { return PAIR && c.r.n * a.G - c.b * RB > TR ? 2 : 1; };

    if (warp < 8) {
        if (warp == 0 || warp == 3) {
            // ============================================================ loads
            // Warp 0 the keys, warp 3 the values and the scales: an issue of copies is a few hundred
            // cycles, and one warp's for both (1600 of 2400 cycles a unit) lay in the way of the ring
            // of two units: 32 requests of 5 x 8 rows 0.200 -> 0.187 ms.
            const int w = warp == 0 ? 0 : 1;
            // Lane i < 8 has keys 16 i .. 16 i + 15 of the unit; the first lane of a page copies it.
            // A page entry is read LA units before its copies and the page's scales one before, so
            // that neither trip to memory lies between one unit's copies and the next's (0.219 ->
            // 0.200 ms, with pages of 16 0.244 -> 0.207; four prompts of 4096 0.397 -> 0.404).
            constexpr int LA = 2;
            Cur c;                           // of the unit whose entries are read next
            c.start(a, s_place);
            int page[LA], head[LA], ahead = 0;    // of units k .. k + LA - 1
            auto look_up = [&](int &pg, int &h) {
                pg = -1;
                h = 0;
                if (ahead >= units) return;
                const int tok = c.t * UT + 16 * lane;
                if (lane < 8 && tok < c.r.kv) pg = a.table[table_at(a, c.r, c.s) + (tok >> a.page_log2)];
                h = c.h;
                if (++ahead < units) c.next_unit(a);
            };
            auto scales_of = [&](int pg, int h, float &ks, float &vs) {
                ks = 0.f, vs = -1.f;         // a page that is gone
                if (pg >= 0 && pg < a.N) {
                    const int64_t ph = (int64_t)pg * a.Hkv + h;
                    ks = a.ks[ph];
                    vs = a.vs[ph];
                }
            };
            const bool first_of_page = lane < 8 && (16 * lane & (P - 1)) == 0;
#pragma unroll
            for (int i = 0; i < LA; ++i) look_up(page[i], head[i]);
            float ks = 0.f, vs = 0.f, ks1 = 0.f, vs1 = 0.f;
            if (w == 1) scales_of(page[0], head[0], ks, vs);
            bool ok = true;
            int x = w;
#pragma unroll 1
            for (int k = 0; k < units; ++k, x += 2) {
                const bool there = page[0] >= 0 && page[0] < a.N, leader = there && first_of_page;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, leader)) * (uint32_t)(P * D);
                const int64_t at = (((int64_t)page[0] * a.Hkv + head[0]) << a.page_log2) * D;
                if (w == 1) scales_of(page[1], head[1], ks1, vs1);
#pragma unroll
                for (int i = 0; i + 1 < LA; ++i) page[i] = page[i + 1], head[i] = head[i + 1];
                look_up(page[LA - 1], head[LA - 1]);
                const int sl = x % NRAW;
                if (x >= NRAW && !(ok = warp_wait(B_RAWFREE + sl, (uint32_t)(x / NRAW - 1)))) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(B_RAWFULL + sl), bytes);
                __syncwarp();
                if (leader)
                    bulk_load(sb + L::OFF_RAW + (uint32_t)sl * L::RAW + (uint32_t)(16 * lane * D), (w ? a.vc : a.kc) + at,
                              (uint32_t)(P * D), bar(B_RAWFULL + sl));
                if (w == 0) continue;
                // the scales: their slot is free, since the values of NSC units ago have been used
                const unsigned gone = __ballot_sync(0xffffffffu, lane < 8 && !there);
                vs = fminf(fmaxf(vs, kv8::kVsMin), kv8::kVsMax);
                if (lane < 8)
                    s_sc[(k % NSC) * 8 + lane] = there ? make_float4(ks, vs, __log2f(vs), __fdividef(1.f, vs)) : make_float4(0.f, -1.f, 0.f, 0.f);
                if (lane == 0) s_gone[k % NSC] = gone != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_SC + k % NSC));
                ks = ks1, vs = vs1;
            }
            // Leave no copy in flight.  Whoever gives up may do so after this warp's last look, so
            // it waits on every path; all but the last few have landed long ago.
            if (lane == 0)
                for (int y = max(w, x - NRAW); y < x; y += 2)
                    mbar_wait(bar(B_RAWFULL + y % NRAW), (uint32_t)(y / NRAW) & 1u, kCleanupLimitNs);
        } else if (warp <= (PAIR ? 2 : 1)) {
            // ============================================================ products
            // PAIR: warp 1 + t issues tile t's, so that a tile waits for its own softmax only; else
            // warp 1 both buffers'.  The whole warp walks the loop, so that the descriptors stay in
            // uniform registers; one elected lane issues.
            constexpr uint32_t id_s = idesc_f16(TR, UT, false), id_o = idesc_f16(TR, D, true);
            bool ok = tmem == 0, issued = false;     // all of the TMEM is ours: its base is 0
            auto give_up = [&]() {
                ok = false;
                s_abort = 1;
                atomicOr(&g_device_error_word, kDevErrTimeout);
            };
            if (!ok) give_up();
            // scores of unit k into buffer b from query tile q; gives the key slot back
            auto scores = [&](int b, int q, int k) {
                tc_fence_after();
                const uint64_t dq = sdesc_sw128(sb + L::OFF_Q + (uint32_t)q * NSL * SLAB, 16, 1024);
                const uint64_t dk = sdesc_sw128(sb + L::OFF_CV + (uint32_t)((2 * k) % NCV) * L::CV, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (uint32_t)(kk >> 2) * SLAB + (uint32_t)(kk & 3) * 32;
                        mma_bf16(TM_S + 128u * b, sdesc_add(dq, off), sdesc_add(dk, off), id_s, kk > 0);
                    }
                    mma_commit(bar(B_S + b));
                    mma_commit(bar(B_CVFREE + (2 * k) % NCV));
                }
                __syncwarp();
                issued = true;
            };
            // the weights of a half (h = 1: keys 64 on, which come first) of buffer b with unit k's
            // values onto its sums
            auto sums = [&](int b, int k, int h, bool fresh) {
                tc_fence_after();
                const uint64_t dv = sdesc_sw128(sb + L::OFF_CV + (uint32_t)((2 * k + 1) % NCV) * L::CV, SLAB, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16_ts(TM_O + 128u * b, TM_S + 128u * b + kP + 32u * h + 8u * kk,
                                   sdesc_add(dv, (4 * h + kk) * 2048), id_o, (!fresh || h == 0 || kk > 0) ? 1u : 0u);
                    if (h == 1) mma_commit(bar(B_U + b));
                }
                __syncwarp();
            };
            // after the second half: gives the value slot back; last: the item's last sums here
            auto sums_done = [&](int b, int k, bool last) {
                if (elect_one()) {
                    mma_commit(bar(B_CVFREE + (2 * k + 1) % NCV));
                    if (last) mma_commit(bar(B_O + b));
                }
                __syncwarp();
            };
            auto just_free = [&](int x) {      // a unit without rows in this tile
                ok = ok && warp_wait(B_CVFULL + x % NCV, (uint32_t)(x / NCV));
                if (ok && lane == 0) mbar_arrive(bar(B_CVFREE + x % NCV));
                __syncwarp();
            };
            if constexpr (PAIR) {
                const int t = warp - 1;
                Cur c, n;                // the unit whose second product is next, and the one after it
                c.start(a, s_place);
                n = c;
                uint32_t nq = 0, np = 0;         // items and units of this tile so far
                // unit k, at n; keys: known to be widened
                auto next_scores = [&](int k, bool fresh, bool keys) {
                    if (t < tiles_of(n)) {
                        if (fresh || !keys)
                            ok = ok && warp_wait3(B_CVFULL + (2 * k) % NCV, (uint32_t)(2 * k / NCV), fresh ? B_Q + t : -1, nq, -1, 0);
                        nq += fresh;
                        if (ok) scores(t, t, k);
                    } else {
                        just_free(2 * k);
                    }
                };
                next_scores(0, true, false);
                // a limit of zero: the next wait has run out before it begins, whatever is there, and
                // the others' that depend on it do
                if (a.limit_ns == 0) give_up();
#pragma unroll 1
                for (int k = 0; ok && k < units; ++k) {
                    const bool last = c.t + 1 == c.nt || k + 1 == units, first = c.t == 0 || k == 0;
                    const int xv = 2 * k + 1;
                    const bool mine = t < tiles_of(c);
                    bool keys = false;
                    if (k + 1 < units) n.next_unit(a);
                    if (mine) {
                        ok = warp_wait3(B_PU + t, np, B_CVFULL + xv % NCV, (uint32_t)(xv / NCV), -1, 0);
                        if (ok) sums(t, k, 1, first);
                        // one look at the next keys on the way
                        const int xk = 2 * k + 2;
                        const bool look = lane == 1 && mbar_test_wait(bar(B_CVFULL + xk % NCV), (uint32_t)(xk / NCV) & 1u);
                        ok = ok && warp_wait(B_P + t, np++);
                        if (!ok) break;
                        sums(t, k, 0, first);
                        sums_done(t, k, last);
                        keys = __any_sync(0xffffffffu, look);
                    } else {
                        just_free(xv);
                    }
                    if (k + 1 < units) next_scores(k + 1, n.t == 0, keys);
                    c = n;
                }
            } else {
                Cur c, n;                // units k (second product) and k + 2 (first)
                c.start(a, s_place);
                n = c;
                uint32_t nq = 0;
                auto next_scores = [&](int k) {      // n is at unit k
                    const bool fresh = k == 0 || n.t == 0;
                    ok = ok && warp_wait3(B_CVFULL + (2 * k) % NCV, (uint32_t)(2 * k / NCV), fresh ? B_Q : -1, nq, -1, 0);
                    nq += fresh;
                    if (ok) scores(k & 1, 0, k);
                    n.next_unit(a);
                };
                // Of units up to the second after k.  NC > 1: of unit k + 1's item only, since the next
                // item's queries are staged when this one's sums have been read.
                int scored = 0;
                auto more_scores = [&](int k) {      // c is at unit k + 1
                    while (ok && scored < units && scored <= k + 2 &&
                           (NC == 1 || (n.s == c.s && n.h == c.h && n.b == c.b)))
                        next_scores(scored++);
                };
                more_scores(-1);
                if (a.limit_ns == 0) give_up();      // (see above)
                int k0 = 0;              // the item's first unit
#pragma unroll 1
                for (int k = 0; ok && k < units; ++k) {
                    const int b = k & 1, xv = 2 * k + 1, k1 = min(units, k + c.nt - c.t);   // the item's end here
                    ok = warp_wait3(B_PU + b, (uint32_t)(k >> 1), B_CVFULL + xv % NCV, (uint32_t)(xv / NCV), -1, 0);
                    if (ok) sums(b, k, 1, k - k0 < 2);
                    ok = ok && warp_wait(B_P + b, (uint32_t)(k >> 1));
                    if (!ok) break;
                    sums(b, k, 0, k - k0 < 2);
                    sums_done(b, k, k + 2 >= k1);
                    c.next_unit(a);
                    if (c.t == 0) k0 = k + 1;
                    more_scores(k);
                }
            }
            if (issued) {   // let this warp's products land before the TMEM goes away, on every path
                if (elect_one()) {
                    mma_commit(bar(B_DRAIN + warp - 1));
                    mbar_wait(bar(B_DRAIN + warp - 1), 0u, kCleanupLimitNs);
                }
                __syncwarp();
            }
        } else if (warp >= 4) {
            // ============================================================ widening
            // Two warps widen the keys, two the values, so that one pair's waits lie under the
            // other's work.  A thread takes 8 codes of a row to 16 bytes of halves: reads and
            // swizzled writes both fall on distinct banks, a thread's rows keep its place in the
            // swizzle, and eight reads are in flight at once.
            Cur c;
            c.start(a, s_place);
            const int w = (warp - 4) >> 1, ct = tid & 63;                // keys or values
            constexpr int PPR = D / 8, RPI = 64 / PPR, IT = UT / RPI, NB = 8;   // pieces a row, rows a step, steps, batch
            const int row0 = ct / PPR, piece = ct % PPR;
            const uint32_t src0 = sb + L::OFF_RAW + (uint32_t)ct * 8;
            const uint32_t dst0 = sb + L::OFF_CV + (uint32_t)(piece >> 3) * SLAB + (uint32_t)row0 * 128u;
            const uint32_t sw0 = ((uint32_t)(piece & 7) ^ (uint32_t)(row0 & 7)) << 4;
            bool ok = true;
#pragma unroll 1
            for (int k = 0, x = w; k < units; ++k, x += 2) {
                const int rs = x % NRAW, cs = x % NCV;
                ok = warp_wait3(B_RAWFULL + rs, (uint32_t)(x / NRAW), x >= NCV ? B_CVFREE + cs : -1, (uint32_t)(x / NCV - 1),
                                w == 1 ? B_SC + k % NSC : -1, (uint32_t)(k / NSC));
                if (!ok) break;
                const uint32_t src = src0 + (uint32_t)rs * L::RAW, dst = dst0 + (uint32_t)cs * L::CV;
                // value codes of places without a cached token: zero, so that no stale NaN
                // meets a zero weight (stale keys only reach scores that are masked)
                const int left = w == 0 ? UT : c.r.kv - c.t * UT;
                const bool holes = w == 1 && s_gone[k % NSC];
                const bool plain = left >= UT && !holes;
#pragma unroll 1
                for (int i0 = 0; i0 < IT; i0 += NB) {
                    uint32_t u[NB][2];
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(u[i][0]), "=r"(u[i][1])
                                     : "r"(src + (uint32_t)(i0 + i) * 512u));
                    if (!plain) {
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const int row = row0 + (i0 + i) * RPI;
                            if (row >= left || (holes && s_sc[(k % NSC) * 8 + (row >> 4)].y < 0.f)) u[i][0] = u[i][1] = 0;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        uint32_t h0, h1, h2, h3;
                        decode4_h<KV>(u[i][0], h0, h1);
                        decode4_h<KV>(u[i][1], h2, h3);
                        // the row's place in the swizzle moves with a step's rows (4 or 8)
                        const uint32_t sw = sw0 ^ (uint32_t)((((i0 + i) * RPI) & 7) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (uint32_t)((i0 + i) * RPI) * 128u + sw),
                                     "r"(h0), "r"(h1), "r"(h2), "r"(h3)
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(B_RAWFREE + rs));
                    mbar_arrive(bar(B_CVFULL + cs));
                }
                c.next_unit(a);
            }
        }
    } else {
        // ================================================================ softmax of buffer b
        const int b = (warp - 8) >> 2, qd = warp & 3;
        const int row = 32 * qd + lane, copy = PAIR ? 0 : 32 * qd / RB;   // of the tile; of the item's rows
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
        const uint32_t ts = tl + TM_S + 128u * b, to = tl + TM_O + 128u * b;
        float2 *s_ml = reinterpret_cast<float2 *>(sm + L::OFF_ML);
        Cur c;
        c.start(a, s_place);
        bool ok = true;
        uint32_t ns = 0, no = 0, no1 = 0, nx = 0, items = 0;   // units and items of this buffer (and of
                                                       // the other's sums), items of the CTA
        int k = 0;                            // unit of the CTA
        typename A::Row r;
        float cs = 0.f;
        // this buffer's rows of the item at c: their place, and their queries for the products.  The
        // one-tile form has one tile of queries, which buffer 0's warps stage and whose factors
        // they leave for buffer 1's.
        const int tile_row0 = PAIR ? b * TR + 32 * qd : 32 * qd % RB;
        uint8_t *const qt = sm + L::OFF_Q + (uint32_t)(PAIR ? b : 0) * NSL * SLAB;
        bool begun = false;                   // the next item's copies are on their way
        auto enter_item = [&]() {
            r = tile_row<RB>(a, c, tile_row0 + lane);
            if (PAIR || b == 0) {
                if (!begun) begin_queries<D, RB>(a, c, tile_row0, qd, smem_u32(qt));
                begun = false;
                cs = end_queries<D>(a, qd, qt, s_fac);
                if (!PAIR && lane == 0) s_cs[qd] = cs;
                if (!PAIR && __float_as_int(cs) < 0) *fac_of(s_fac + TR) = *fac_of(s_fac);     // and for buffer 1
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_Q + (PAIR ? b : 0)));
            }
        };
        bool mine_item = !PAIR || b < tiles_of(c);
        if (mine_item) enter_item();
        // PAIR: the next item's queries, once this one's last scores are there (the tile is free)
        auto begin_next = [&]() {
            if (!PAIR || k + (c.nt - c.t) >= units) return;
            Cur n = c;
            n.next_of_item(a);
            if (b >= tiles_of(n)) return;
            begin_queries<D, RB>(a, n, tile_row0, qd, smem_u32(qt));
            begun = true;
        };
#pragma unroll 1
        while (k < units && ok) {
            const int mine = min(c.nt - c.t, units - k);      // the CTA's units of this item
            const bool first = c.t == 0, last = c.t + mine == c.nt, whole = first && last;
            const int t0 = c.t;
            if (tid == 256) {
                // the CTA's entry: an item that begins here and ends elsewhere (its last)
                if (first && !last)
                    a.entry[blockIdx.x] = make_int4(cta_of(s_place, u0 + k + c.nt - 1, s_place.i0 + items), c.s, c.h, c.b);
                else if (k + mine == units)
                    a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
            }
            float M = -INFINITY, l = 0.f;
            if (mine_item) {
                const int j0 = PAIR ? 0 : (k ^ b) & 1, dj = PAIR ? 1 : 2;   // not PAIR: units of this parity
                RowUnit<GR> u;
                u.cs = cs;
                u.fac = s_fac;
                const bool any_live = __any_sync(0xffffffffu, r.live);
                bool gone = false;
                auto scales_of = [&](int kk) {     // of unit kk, whose scale slot has been waited for
                    u.sc = s_sc + (kk % NSC) * 8;
                    if constexpr (PAIR && GR == 1) u.held[0] = u.sc[0], u.held[1] = u.sc[4];
                    if constexpr (NC == 2 && GR == 1) u.held[0] = u.held[1] = u.sc[4 * copy];
                    gone = s_gone[kk % NSC];
                };
#pragma unroll 1
                for (int j = j0; j < mine && ok; j += dj) {
                    const int kk = k + j;
                    ok = warp_wait(B_S + b, ns++);
                    // An item's first unit: the scores came first, so a tile that sat out items is now
                    // at this unit and the scale slot's phase is the one before or after its publication.
                    if (ok && j == j0 && any_live) {
                        ok = warp_wait(B_SC + kk % NSC, (uint32_t)(kk / NSC));
                        scales_of(kk);
                    }
                    if (!ok) break;
                    if (j + dj >= mine) begin_next();
                    if (!PAIR && b == 1 && j == j0) cs = u.cs = s_cs[qd];     // staged before these scores
                    if (!any_live) {      // a warp without rows: its weights are never looked at
                        if (!PAIR && b == 1 && j == j0 && items > 0 && !(ok = warp_wait(B_OFREE, items - 1))) break;
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(B_PU + b));
                            mbar_arrive(bar(B_P + b));
                        }
                        continue;
                    }
                    tc_fence_after();
                    u.see = r.lim - (t0 + j) * UT;
                    u.part = __any_sync(0xffffffffu, u.see < UT) || gone || __float_as_int(u.cs) < 0;
                    ok = softmax_unit<D, GR, PAIR, NC>(ts, to, u, copy, j > j0, M, l, [&](int h) {
                        // the weights let buffer 1's sums be written again: not before buffer 0's
                        // warps have read those of the item before
                        if (!PAIR && h == 1 && b == 1 && j == j0 && items > 0 && !warp_wait(B_OFREE, items - 1)) return false;
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar((h == 1 ? B_PU : B_P) + b));
                        return true;
                    }, [&]() {
                        const bool there = warp_wait(B_U + b, ns - 1);
                        tc_fence_after();
                        return there;
                    });
                    if (!ok) break;
                    // the next unit's scale slot, while its scores are made
                    if (j + dj < mine) {
                        ok = warp_wait(B_SC + (kk + dj) % NSC, (uint32_t)((kk + dj) / NSC));
                        scales_of(kk + dj);
                    }
                }
            }
            // ---- the item's sums, after the next item's queries are on their way
            const typename A::Row done = r;
            const int64_t slot = ((int64_t)blockIdx.x * 2 + (first ? 1 : 0)) * RB + tile_row0 + lane;
            const bool had = mine_item;
            const int had0 = PAIR ? mine : (mine + 1 - (k & 1)) >> 1, had1 = PAIR ? mine : (mine + (k & 1)) >> 1;
            k += mine;
            c.next_of_item(a);
            auto next_item_queries = [&]() {
                mine_item = k < units && (!PAIR || b < tiles_of(c));
                if (ok && mine_item) enter_item();
            };
            if constexpr (PAIR) {
                next_item_queries();
                if (had) {
                    ok = ok && warp_wait(B_O + b, no++);
                    if (!ok) break;
                    tc_fence_after();
                    const auto end = end_row<D>(a, done, whole, M, l);
#pragma unroll 1
                    for (int cb = 0; cb < D / 32; ++cb) {
                        float o[32];
                        tmem_ld32(to + 32u * cb, o);
                        tmem_wait_ld();
                        write_chunk<D, RB>(a, done, whole, slot, cb, end, o);
                    }
                    write_stats(a, done, whole, slot, M, l);
                    tc_fence_before();
                }
            } else if (b == 1) {
                // hand M and l over (the item before's have been read); buffer 0's warps join the sums
                if (had1 == 0 && items > 0) ok = ok && warp_wait(B_OFREE, items - 1);
                if (ok) {
                    s_ml[row] = make_float2(M, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_ML));
                }
                next_item_queries();
            } else if constexpr (NC > 1) {
                // The copies' sums are joined through the query tile, 32 columns at a time in two
                // places in turn; copy 0 writes them.  Its queries are read no more: all scores are done.
                ok = ok && warp_wait(B_ML, items);
                if (ok && had0 > 0) ok = warp_wait(B_O + 0, no++);
                if (ok && had1 > 0) ok = warp_wait(B_O + 1, no1++);
                if (!ok) break;
                tc_fence_after();
                auto meet = [&]() {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_X));
                    return warp_wait(B_X, nx++);
                };
                const float2 ml = s_ml[row];
                const float Mt = fmaxf(M, ml.x);
                const float w0 = M == Mt ? 1.f : part_weight(M, Mt), w1 = ml.x == Mt ? 1.f : part_weight(ml.x, Mt);
                s_ml[row] = make_float2(Mt, l * w0 + ml.y * w1);
                if (!(ok = meet())) break;
                float Ma = -INFINITY, la = 0.f;
#pragma unroll
                for (int q = 0; q < NC; ++q) Ma = fmaxf(Ma, s_ml[q * RB + row % RB].x);
#pragma unroll
                for (int q = 0; q < NC; ++q) {
                    const float2 x = s_ml[q * RB + row % RB];
                    la = fmaf(x.x == Ma ? 1.f : part_weight(x.x, Ma), x.y, la);
                }
                const float f = Mt == Ma ? 1.f : part_weight(Mt, Ma);
                const auto end = end_row<D>(a, done, whole, Ma, la);
#pragma unroll 1
                for (int cb = 0; cb < D / 32; ++cb) {
                    float o[32], o1[32];
                    tmem_ld32(to + 32u * cb, o);          // a buffer without sums is read, not used
                    tmem_ld32(to + 128u + 32u * cb, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = ((had0 > 0 ? o[e] * w0 : 0.f) + (had1 > 0 ? o1[e] * w1 : 0.f)) * f;
                    // row x of the copies after the first, 16-byte pieces spread over the banks
                    auto piece = [&](int x, int e) {
                        return reinterpret_cast<float4 *>(sm + L::OFF_Q + (cb & 1) * L::XR + x * 128 + ((e ^ (x & 7)) << 4));
                    };
                    if (copy > 0)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *piece(row - RB, e) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    if (!(ok = meet())) break;
                    if (copy == 0) {
#pragma unroll 1
                        for (int q = 0; q < NC - 1; ++q)
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 x = *piece(q * RB + row, e);
                                o[4 * e] += x.x, o[4 * e + 1] += x.y, o[4 * e + 2] += x.z, o[4 * e + 3] += x.w;
                            }
                        write_chunk<D, RB>(a, done, whole, slot, cb, end, o);
                    }
                }
                if (!ok) break;
                if (copy == 0) write_stats(a, done, whole, slot, Ma, la);
                tc_fence_before();
                if (!(ok = meet())) break;            // copy 0 has read what the others left
                if (lane == 0) mbar_arrive(bar(B_OFREE));
                next_item_queries();
            } else {
                // the other buffer's scores are done once its M and l are here (or it had none), so
                // the query tile may be written again
                ok = ok && warp_wait(B_ML, items);
                if (!ok) break;
                const float2 ml = s_ml[row];
                next_item_queries();
                if (had0 > 0) ok = ok && warp_wait(B_O + 0, no++);
                if (had1 > 0) ok = ok && warp_wait(B_O + 1, no1++);
                if (!ok) break;
                tc_fence_after();
                float Mt = fmaxf(M, ml.x);
                const float w0 = M == Mt ? 1.f : part_weight(M, Mt), w1 = ml.x == Mt ? 1.f : part_weight(ml.x, Mt);
                float lt = l * w0 + ml.y * w1;
                const auto end = end_row<D>(a, done, whole, Mt, lt);
#pragma unroll 1
                for (int cb = 0; cb < D / 32; ++cb) {
                    float o[32], o1[32];
                    tmem_ld32(to + 32u * cb, o);          // a buffer without sums is read, not used
                    tmem_ld32(to + 128u + 32u * cb, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = (had0 > 0 ? o[e] * w0 : 0.f) + (had1 > 0 ? o1[e] * w1 : 0.f);
                    write_chunk<D, RB>(a, done, whole, slot, cb, end, o);
                }
                write_stats(a, done, whole, slot, Mt, lt);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_OFREE));
            }
            ++items;
        }
    }
    if (warp >= 8) {      // and a softmax warp's queries and weights, where it gave up under them
        asm volatile("cp.async.wait_all;" ::: "memory");
        tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (s_abort && tid == 0) a.entry[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (warp == 1) tmem_dealloc(tmem, TM_COLS);
    grid_launch_dependents();
}

// What the rows' 32-byte stores go to.
uintptr_t stored_at(const AttnArgs &a) { return reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.part_o); }
template <bool F>
uintptr_t stored_at(const SharedArgs<F> &a) { return stored_at(static_cast<const AttnArgs &>(a)) | reinterpret_cast<uintptr_t>(a.pre_o); }
template <Kv8 KV, int D, bool PAIR, int NC, int GR, class A>
cudaError_t launch_tile_g(A &a, void *ws, int ctas, int64_t rows, cudaStream_t s) {
    using L = tl::Lay<D, PAIR, NC>;
    place_parts(a, ws, ctas, L::RB);
    a.wide = (stored_at(a) & 31) == 0;
    auto kernel = kv8_tile_kernel<KV, D, PAIR, NC, GR, A>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kernel, L::SMEM, allowed);
    if (e != cudaSuccess) return e;
    attended.store(true, std::memory_order_relaxed);
    if ((e = launch_after(kernel, dim3((unsigned)ctas), tl::NT, L::SMEM, s, a)) != cudaSuccess) return e;
    return launch_merge<__nv_bfloat16, D, L::RB>(a, rows, s);
}
template <Kv8 KV, int D, bool PAIR, int NC, class A>
cudaError_t launch_tile_f(A &a, void *ws, int ctas, int64_t rows, cudaStream_t s) {
    return a.page_log2 >= 6 ? launch_tile_g<KV, D, PAIR, NC, 1>(a, ws, ctas, rows, s)
                            : launch_tile_g<KV, D, PAIR, NC, 4>(a, ws, ctas, rows, s);
}

// Pairs of tiles where a request may have more rows than one tile (96 rows, 32 requests on 1000 to
// 16 k keys: one tile 0.108 ms, pairs 0.138; 4 on 4000 keys 28.6 and 27.9 us); where they fill a
// half or a quarter of one, that many copies of them (40 rows, 32 on 1000 to 16 k: two copies 0.092
// ms, one 0.104; 24 rows: four 0.0883, two 0.0890, one 0.100; on 100 to 600 keys, where an item's
// ends weigh more, 26 us with copies and 23 to 24 with one).
template <Kv8 KV, int D, class A>
cudaError_t launch_tile_d(A &a, void *ws, int ctas, int64_t rows, cudaStream_t s) {
    return rows > tl::TR       ? launch_tile_f<KV, D, true, 1>(a, ws, ctas, rows, s)
           : rows > tl::TR / 2 ? launch_tile_f<KV, D, false, 1>(a, ws, ctas, rows, s)
           : rows > tl::TR / 4 ? launch_tile_f<KV, D, false, 2>(a, ws, ctas, rows, s)
                               : launch_tile_f<KV, D, false, 4>(a, ws, ctas, rows, s);
}
template <Kv8 KV, class A>
cudaError_t launch_tile_kv(A &a, int D, void *ws, int64_t rows, cudaStream_t s) {
    const int ctas = sm_count();
    return D == 128 ? launch_tile_d<KV, 128>(a, ws, ctas, rows, s) : launch_tile_d<KV, 64>(a, ws, ctas, rows, s);
}

}  // namespace
}  // namespace gdr
