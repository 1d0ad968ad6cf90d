// gdr_kv8_attn.cuh -- what the two attention kernels over the 8-bit paged cache share: their
// arguments, the division of the work among CTAs, and the partial results of divided items.
//
// Work.  A request's n queries and the G = Hq / Hkv query heads of one cached head form
// n * G rows (row r: query r / G, head r % G), which all read the same keys.  An item is a
// block of RB such rows with the keys its last row sees, in units of UT tokens (an item that
// sees nothing keeps one unit, which writes its zeros).  All units of a call stand in one order
// (request, head, block, tokens), each item's after as much more as its ends cost (E units), and
// that length is divided evenly among the CTAs, whatever the requests' lengths are: of a total
// of w, CTA c of n takes the units that lie in [w c / n, w (c + 1) / n).  Lengths stay on the
// device; every CTA finds its first unit by a prefix sum over the requests.
//
// An item that falls to several CTAs leaves in each an unnormalised partial result (fp32
// sums, the reference exponent and the weight sum of every row) in the CTA's slot 1 (the CTA
// where the item begins) or slot 0 (the ones after it), and the first CTA an entry that the
// merge kernel follows.  The order of the merge is that of the tokens, so results repeat.
#pragma once

#include "gdr_fused_common.cuh"
#include "gdr_kv8.cuh"

#include <algorithm>
#include <atomic>

namespace gdr {
namespace {

namespace kv8 {
// Weights are 2^(x - M + kOff), at most 2^(kOff + kTau): a half holds them, 11 bits of those down to
// 2^-14 and steps of 2^-24 below.  M moves when a score exceeds it by more than kTau.
constexpr float kOff = 14.f, kTau = 1.5f;
constexpr float kVsMin = 9.094947017729282e-13f, kVsMax = 1.099511627776e12f;   // 2^-40, 2^40
// CTAs of the merge that an SM holds (256 threads of 64 registers).  Rows are taken with eight warps
// each while all of them are resident at once (512 rows of 8 x 2 tokens on 6000 keys 24.2 us, with
// a warp each 25.4); beyond, the waves cost more than the shorter walks give (24 tokens on 1000
// keys, 768 rows: 20.7 and 19.5; 56 tokens, 1792 rows: 26.7 and 21.4).
constexpr int kMergeResident = 4;
}  // namespace kv8

struct AttnArgs {
    const void *q;
    int64_t q_stride;
    const float *ks, *vs;
    const int *table, *kv_len, *cu_q;
    float scale_log2;            // |score scale| / ln 2; its sign goes into the queries, so that
    float sign;                  // a larger product is a larger score (cache scales are positive)
    const uint8_t *kc, *vc;
    void *out;
    float *lse;
    float *part_o;               // [CTA][2][RB][D]
    float *part_ml;              // [CTA][2][RB][2]: reference exponent M, weight sum
    int4 *entry;                 // [CTA] {last CTA (-1: no divided item), request, head, block}
    int S, total_q, Hq, Hkv, G, W, page_log2, N;
    int ctas;                    // of the attention kernel
    bool wide;                   // out and part_o are 32-byte aligned
    uint64_t limit_ns;
};

// One request, as every kernel reads it: offsets and lengths are clamped to the tensors.
struct Request {
    int q0, n, kv;
};
__device__ __forceinline__ Request request_of(const AttnArgs &a, int s) {
    Request r;
    r.kv = (int)min((int64_t)max(a.kv_len[s], 0), (int64_t)a.W << a.page_log2);
    if (a.cu_q) {
        r.q0 = min(max(a.cu_q[s], 0), a.total_q);
        r.n = min(max(a.cu_q[s + 1], r.q0), a.total_q) - r.q0;
    } else {
        r.q0 = s;
        r.n = 1;
    }
    return r;
}
// Keys that query i sees, and those that block b of RB rows does (its last row sees the most).
__device__ __forceinline__ int seen_by(const Request &r, int i) { return max(0, min(r.kv, r.kv - r.n + i + 1)); }
template <int RB>
__device__ __forceinline__ int block_end(const AttnArgs &a, const Request &r, int b) {
    return seen_by(r, (min(r.n * a.G, (b + 1) * RB) - 1) / a.G);
}
template <int RB>
__device__ __forceinline__ int blocks_of(const AttnArgs &a, const Request &r) { return (r.n * a.G + RB - 1) / RB; }
template <int UT>
__device__ __forceinline__ int units_of(int end) { return max(1, (end + UT - 1) / UT); }
template <int RB, int UT>
__device__ __forceinline__ int64_t units_of_head(const AttnArgs &a, const Request &r) {
    const int nb = blocks_of<RB>(a, r);
    int64_t u = 0;
    for (int b = 0; b < nb; ++b) u += units_of<UT>(block_end<RB>(a, r, b));
    return u;
}

struct Place {      // a unit: request, head, block of rows, unit of the block's keys
    int s, h, b, t;
    int ctas, extra;         // CTAs with work; units that an item's ends count for
    int64_t u0, u1, i0;      // this CTA's units, the items before the first one's
    int64_t total;           // what is shared: all units, and `extra` for each item
};

// This CTA's units and the place of the first one.  An item costs its units and, for its queries
// and its end, as much as E more; what is divided evenly is the sum of both (the units of an
// item follow its E), or the units alone where a CTA's share would be no more than E.  All NT
// threads call it; `place` is in shared memory and valid after it returns.
template <int RB, int UT, int NT, int E>
__device__ __forceinline__ void find_place(const AttnArgs &a, Place *place, int64_t *s_scan) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = NT / 32;
    struct Sum {
        int64_t u, i;        // units, items
    };
    Sum mine{}, before{}, sum{};
    // what comes before each request of a chunk of NT requests; the last chunk stays in registers
    auto scan = [&](int base) {
        const int s = base + tid;
        mine = Sum{0, 0};
        if (s < a.S) {
            const Request r = request_of(a, s);
            mine.u = units_of_head<RB, UT>(a, r) * a.Hkv;
            mine.i = (int64_t)blocks_of<RB>(a, r) * a.Hkv;
        }
        Sum incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, incl.u, off), i = __shfl_up_sync(0xffffffffu, incl.i, off);
            if (lane >= off) incl.u += u, incl.i += i;
        }
        __syncthreads();
        if (lane == 31) s_scan[2 * warp] = incl.u, s_scan[2 * warp + 1] = incl.i;
        __syncthreads();
        before = Sum{incl.u - mine.u, incl.i - mine.i};
        sum = Sum{0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int64_t u = s_scan[2 * w], i = s_scan[2 * w + 1];
            if (w < warp) before.u += u, before.i += i;
            sum.u += u, sum.i += i;
        }
    };
    Sum all{};
    for (int base = 0; base < a.S; base += NT) {
        scan(base);
        all.u += sum.u, all.i += sum.i;
    }
    const int e = all.u + E * all.i >= (int64_t)(E + 1) * gridDim.x ? E : 0;
    const int64_t total = all.u + e * all.i;
    // fewer units than CTAs: one each, so that the parts of an item lie in consecutive CTAs
    // (as they do with e > 0, when no CTA's share is less than the way from one unit to the next)
    const int64_t ctas = min((int64_t)gridDim.x, max(total, (int64_t)1));
    const int64_t w0 = blockIdx.x < ctas ? total * blockIdx.x / ctas : total;
    const int64_t w1 = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : total;
    if (tid == 0) {
        place->u0 = all.u;
        place->u1 = all.u;
        place->total = total;
        place->ctas = (int)ctas;
        place->extra = e;
    }
    __syncthreads();
    if (w0 < w1) {
        Sum run{};
        for (int base = 0; base < a.S; base += NT) {
            if (a.S > NT) scan(base);
            const int64_t at = run.u + before.u + e * (run.i + before.i), end = at + mine.u + e * mine.i;
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {            // the first unit at or after w0, and after w1
                const int64_t w = k ? w1 : w0;
                if (w < at || w >= end) continue;
                const Request r = request_of(a, base + tid);
                const int64_t per_u = mine.u / a.Hkv, per_i = mine.i / a.Hkv, h = (w - at) / (per_u + e * per_i);
                int64_t rem = w - at - h * (per_u + e * per_i), u = run.u + before.u + h * per_u;
                int b = 0;
                for (;; ++b) {
                    const int n = units_of<UT>(block_end<RB>(a, r, b));
                    if (rem < n + e) break;
                    rem -= n + e;
                    u += n;
                }
                const int t = (int)max(rem - e, (int64_t)0);
                if (k) {
                    place->u1 = u + t;
                } else {
                    place->u0 = u + t;
                    place->i0 = run.i + before.i + h * per_i + b;
                    place->s = base + tid, place->h = (int)h, place->b = b, place->t = t;
                }
            }
            run.u += sum.u, run.i += sum.i;
        }
    }
    __syncthreads();
}

// The CTA that has unit u, which belongs to item i.
__device__ __forceinline__ int cta_of(const Place &p, int64_t u, int64_t i) {
    return (int)(((u + p.extra * (i + 1) + 1) * p.ctas - 1) / p.total);
}

// Moves to the next item: next block, head, request with queries.
template <int RB>
__device__ __forceinline__ void next_item(const AttnArgs &a, int &s, int &h, int &b, Request &r) {
    if (++b < blocks_of<RB>(a, r)) return;
    b = 0;
    if (++h < a.Hkv) return;
    h = 0;
    do {
        if (++s >= a.S) return;
        r = request_of(a, s);
    } while (r.n == 0);
}

// A role's way through this CTA's units.
template <int RB, int UT>
struct Cursor {
    int s, h, b, t, nt, end;     // item, unit, the item's units and keys
    Request r;
    __device__ __forceinline__ void enter(const AttnArgs &a) {
        end = block_end<RB>(a, r, b);
        nt = units_of<UT>(end);
    }
    __device__ __forceinline__ void start(const AttnArgs &a, const Place &p) {
        s = p.s, h = p.h, b = p.b, t = p.t;
        r = request_of(a, s);
        enter(a);
    }
    __device__ __forceinline__ void next_of_item(const AttnArgs &a) {   // past the last item: s = S
        t = 0;
        next_item<RB>(a, s, h, b, r);
        if (s < a.S) enter(a);
    }
    __device__ __forceinline__ void next_unit(const AttnArgs &a) {
        if (++t == nt) next_of_item(a);
    }
};

template <typename E> struct Vec16;   // 16 bytes of E as floats and back
template <> struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float *f) {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *f) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *f) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *f) {
        uint4 u;
        u.x = pack_bf16x2(f[0], f[1]);
        u.y = pack_bf16x2(f[2], f[3]);
        u.z = pack_bf16x2(f[4], f[5]);
        u.w = pack_bf16x2(f[6], f[7]);
        *reinterpret_cast<uint4 *>(p) = u;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(m - ref) for exponents of partial results; 0 for a part that saw nothing.
__device__ __forceinline__ float part_weight(float m, float ref) { return m == -INFINITY ? 0.f : ex2(m - ref); }

// The power of two that brings a row of largest magnitude amax below 2^15, where a half
// keeps 11 bits of everything that counts (bf16 values exactly, down to 2^-29 of the
// largest); 1 for a row of zeros.  With an infinity the least one, which leaves finite values
// finite: they do not count beside it.
__device__ __forceinline__ float row_factor(float amax) {
    const int x = min((int)(__float_as_uint(amax) >> 23) & 255, 254);   // 2^(x - 127) <= amax
    if (amax == 0.f) return 1.f;
    return __uint_as_float((uint32_t)min(268 - x, 253) << 23);   // 2^(14 - (x - 127)); its inverse is normal
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ------------------------------------------------------------------ merge of divided items
// A CTA takes rows of the blockIdx.x-th divided item.  WPR warps take one row, a run of its parts
// each (few rows, many parts: one request of 5 x 8 rows on 4000 keys, 32 parts an item, 57 -> 17
// us for the whole call against a warp that walks the parts of row after row), or one warp takes
// RPW rows at once (many rows, few parts).  A lane weighs a part, then the lanes take the D
// values: eight loads are in flight at once, since each is a trip to the L2.
// ROUND: the grid may be too small for the items and rows that there are (max_q says less than
// the lengths do), and goes round; the loops cost up to 1 us (7 ragged fp32 requests: 22.1 and 23.4 us).
template <typename E, int D, int RB, int WPR, int RPW, bool ROUND>
__global__ void __launch_bounds__(256, kv8::kMergeResident) kv8_merge_kernel(const AttnArgs a) {
    static_assert(WPR == 1 ? !ROUND : RPW == 1, "");
    constexpr int VL = D / 32;
    __shared__ float s_o[WPR > 1 ? 8 : 1][D];
    __shared__ float s_l[8];
    __shared__ uint32_t s_mask[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w0 = warp / WPR * WPR;
    grid_dependency_wait();
    grid_launch_dependents();
    bool again = false;
    auto item = [&](int c0) {
        const int4 en = a.entry[c0];
        if (en.x < 0) return;
        const Request r = request_of(a, en.y);
        const int rows = min(RB, r.n * a.G - en.w * RB), parts = en.x - c0 + 1;
        constexpr int STEP = 8 / WPR * RPW;
#pragma unroll 1
        for (int row0 = blockIdx.y * STEP + warp / WPR * RPW; row0 < rows; row0 += gridDim.y * STEP) {
            // row rr of part p; a row that is not there is read as the last one and not written
            auto slot = [&](int p, int rr) { return ((int64_t)(c0 + p) * 2 + (p == 0 ? 1 : 0)) * RB + min(row0 + rr, rows - 1); };
            float ref[RPW], l[RPW], o[RPW][VL];
            float2 ml[RPW];
#pragma unroll
            for (int rr = 0; rr < RPW; ++rr) {
                ref[rr] = -INFINITY;
                l[rr] = 0.f;
#pragma unroll
                for (int e = 0; e < VL; ++e) o[rr][e] = 0.f;
            }
            for (int p = lane; p - lane < parts; p += 32)
#pragma unroll
                for (int rr = 0; rr < RPW; ++rr) {
                    const float2 x = p < parts ? *reinterpret_cast<const float2 *>(a.part_ml + 2 * slot(p, rr)) : make_float2(-INFINITY, 0.f);
                    ref[rr] = fmaxf(ref[rr], x.x);
                    if (p == lane) ml[rr] = x;
                }
            float M[RPW];
#pragma unroll
            for (int rr = 0; rr < RPW; ++rr) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) ref[rr] = fmaxf(ref[rr], __shfl_xor_sync(0xffffffffu, ref[rr], off));
                M[rr] = ref[rr] == -INFINITY ? 0.f : ref[rr];
            }
            const int per = (parts + WPR - 1) / WPR, end = min(parts, (warp - w0 + 1) * per);
            for (int p0 = (warp - w0) * per; p0 < end; p0 += 32) {
                const int n = min(32, end - p0);
                float w[RPW];
#pragma unroll
                for (int rr = 0; rr < RPW; ++rr) {
                    if (p0 > 0) ml[rr] = *reinterpret_cast<const float2 *>(a.part_ml + 2 * slot(min(p0 + lane, parts - 1), rr));
                    // a part without an exponent weighs 0; if its sums are NaN (all its scores are) they stay NaN
                    w[rr] = part_weight(ml[rr].x, M[rr]);
                    if (lane < n) l[rr] = fmaf(w[rr], ml[rr].y, l[rr]);
                }
#pragma unroll(8 / RPW)
                for (int j = 0; j < n; ++j)
#pragma unroll
                    for (int rr = 0; rr < RPW; ++rr) {
                        const float wj = __shfl_sync(0xffffffffu, w[rr], j);
                        const float *src = a.part_o + slot(p0 + j, rr) * D + lane * VL;
                        if constexpr (VL == 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(src);
                            o[rr][0] = fmaf(wj, x.x, o[rr][0]), o[rr][1] = fmaf(wj, x.y, o[rr][1]);
                            o[rr][VL - 2] = fmaf(wj, x.z, o[rr][VL - 2]), o[rr][VL - 1] = fmaf(wj, x.w, o[rr][VL - 1]);
                        } else {
                            const float2 x = *reinterpret_cast<const float2 *>(src);
                            o[rr][0] = fmaf(wj, x.x, o[rr][0]), o[rr][1] = fmaf(wj, x.y, o[rr][1]);
                        }
                    }
            }
#pragma unroll
            for (int rr = 0; rr < RPW; ++rr)
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], off);
            if constexpr (WPR > 1) {
                if (ROUND && again) __syncthreads();
                again = true;
                if (lane == 0) s_l[warp] = l[0];
#pragma unroll
                for (int e = 0; e < VL; ++e) s_o[warp][lane * VL + e] = o[0][e];
                __syncthreads();
                if (warp != w0) {
                    if constexpr (ROUND) continue;
                    return;
                }
                l[0] = 0.f;
#pragma unroll
                for (int w = 0; w < WPR; ++w) l[0] += s_l[w0 + w];
#pragma unroll
                for (int e = 0; e < VL; ++e) {
                    o[0][e] = 0.f;
#pragma unroll
                    for (int w = 0; w < WPR; ++w) o[0][e] += s_o[w0 + w][lane * VL + e];
                }
            }
#pragma unroll
            for (int rr = 0; rr < RPW; ++rr) {
                const int row = row0 + rr, at = en.w * RB + row;
                if (row >= rows) break;
                const float inv = l[rr] == 0.f ? 0.f : 1.f / l[rr];
                const int64_t orow = (int64_t)(r.q0 + at / a.G) * a.Hq + en.z * a.G + at % a.G;
#pragma unroll
                for (int e = 0; e < VL; ++e) {
                    if constexpr (sizeof(E) == 4)
                        static_cast<float *>(a.out)[orow * D + lane * VL + e] = o[rr][e] * inv;
                    else
                        static_cast<__nv_bfloat16 *>(a.out)[orow * D + lane * VL + e] = __float2bfloat16_rn(o[rr][e] * inv);
                }
                if (a.lse && lane == 0)
                    a.lse[orow] = l[rr] == 0.f ? -INFINITY : (M[rr] - kv8::kOff + log2f(l[rr])) * 0.693147180559945f;
            }
            if constexpr (!ROUND) return;
        }
    };
    // the blockIdx.x-th entry that has an item (ROUND: and every gridDim.x-th after it), 1024 entries
    // at a time; with a CTA for every entry, its own
    const bool own = gridDim.x == a.ctas;
    for (int base = 0, before = 0, next = blockIdx.x; base < a.ctas; base += 1024) {
        int incl = 0;
        if (!own) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = base + 256 * i + threadIdx.x;
                const unsigned m = __ballot_sync(0xffffffffu, c < a.ctas && a.entry[min(c, a.ctas - 1)].x >= 0);
                if (lane == 0) s_mask[8 * i + warp] = m;
            }
            __syncthreads();
            incl = __popc(s_mask[lane]);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            incl += before;
        }
#pragma unroll 1
        while (true) {
            int c0 = next;
            if (!own) {
                const unsigned past = __ballot_sync(0xffffffffu, incl > next);
                if (past == 0) break;
                const int g = __ffs(past) - 1;
                const unsigned m = s_mask[g];
                c0 = base + 32 * g + (int)__fns(m, 0, next - (__shfl_sync(0xffffffffu, incl, g) - __popc(m)) + 1);
            }
            item(c0);
            if (own || !ROUND) return;
            next += gridDim.x;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
    }
}

// SMs of the current device, asked once a device.
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    const bool in = dev >= 0 && dev < 64;
    if (in && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    if (in) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}
// A launch that may start while the kernel before it in the stream ends (both wait before they
// read what another kernel writes).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// CTAs for as many items as can be divided among the attention's `a.ctas` (each at most one, and
// there are no more than the requests' blocks of rows), or for every entry where that is not
// much more: looking for the item takes 1.5 us.  `rows` goes by max_q; where the lengths could be
// more than that, the wide form goes round and the other has CTAs for what they could be.
template <typename E, int D, int RB>
cudaError_t launch_merge(const AttnArgs &a, int64_t rows, cudaStream_t s) {
    constexpr int RPW = RB >= 16 ? 2 : 1;
    const int64_t all = (int64_t)a.total_q * a.G;      // rows of all requests
    const int64_t most = std::min(rows, (int64_t)RB), could = std::min(all, (int64_t)RB);
    const int64_t limit = (all + (int64_t)a.S * (RB - 1)) / RB, blocks = std::min((int64_t)a.S * ((rows + RB - 1) / RB), limit);
    const int64_t items = 2 * blocks * a.Hkv < a.ctas ? blocks * a.Hkv : a.ctas;
    const bool every = items == a.ctas || blocks == limit;
    const unsigned x = (unsigned)items, all_x = (unsigned)std::min(limit * a.Hkv, (int64_t)a.ctas);
    const unsigned wide = (unsigned)most, y = (unsigned)((could + 8 * RPW - 1) / (8 * RPW));
    if (items * most <= kv8::kMergeResident * sm_count()) {
        if (every && most == could) return launch_after(kv8_merge_kernel<E, D, RB, 8, 1, false>, dim3(x, wide), 256, 0, s, a);
        return launch_after(kv8_merge_kernel<E, D, RB, 8, 1, true>, dim3(x, wide), 256, 0, s, a);
    }
    return launch_after(kv8_merge_kernel<E, D, RB, 1, RPW, false>, dim3(every ? x : all_x, y), 256, 0, s, a);
}

// Entries, then {M, l}, then the sums.
size_t part_bytes(int ctas, int RB, int D) {
    return (size_t)ctas * (sizeof(int4) + (size_t)2 * RB * (2 + D) * sizeof(float));
}
void place_parts(AttnArgs &a, void *ws, int ctas, int RB) {
    a.ctas = ctas;
    a.entry = static_cast<int4 *>(ws);
    a.part_ml = reinterpret_cast<float *>(a.entry + ctas);
    a.part_o = a.part_ml + (size_t)ctas * 2 * RB * 2;
}

// The kernel's shared-memory limit, raised once a device (`done`: one flag a kernel).
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace
}  // namespace gdr
