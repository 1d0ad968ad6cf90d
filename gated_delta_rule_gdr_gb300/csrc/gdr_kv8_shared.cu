// gdr_kv8_shared.cu -- attention over the 8-bit paged cache for requests that share a prefix: which pages
// the requests of a group have in common (gdr_kv8_shared_plan), and the attention, which reads these once
// for all of the group's queries (gdr_kv8_attn_shared).
//
// A softmax over two sets of keys is the two sets' sums with a joint reference: with sums O_i, l_i of
// weights 2^(x - M_i),  O = sum_i 2^(M_i - M) O_i,  l likewise,  out = O / l.  So the keys that all queries
// of a group see need no query's own mask, and their rows (queries x heads of a cached head) can be
// items of any shape: the group is a request of its own to the attention kernels.  Two passes:
//   first   the groups' common pages, for all of their rows: many rows a cached head, so the tile
//           kernel for all but small groups; every row's sums stay in the workspace as fp32
//   second  every request's own pages, as in gdr_kv8_attn; where a row's sums are complete (in the
//           kernel or its merge) the first pass's are joined to them and the output is rounded once
//
// Bound: the common pages' codes once a group and the others' once, or, with many rows, the products.
// Measured: 256 single tokens of 8 heads a cached head, four groups with 17 to 32 k common tokens and up to
// 2000 of their own (372 MB, 107 GFLOP: 56 us either way) 237 us, gdr_kv8_attn 928: the tile kernel 154 (four
// of eleven blocks of 256 rows are half empty; 2.6 us a block and 128 keys), its merge 10, the own tokens 72
// (270 MB, 1000 keys an item: its ends weigh; 3.8 TB/s), their merge 7.  24 questions of up to 200 tokens of 4 heads a
// cached head on 20 k (595 GFLOP, 310 us) 647 us, gdr_kv8_attn 800: 1000 TFLOP/s in the first pass (570 us),
// the rest the questions' own tiles and 60 MB of sums on their way.
// The plan: 256 requests in 8 groups 3.5 us, 1000 rows of 4096 entries (16.4 MB) 7.4 us, two launches; every
// CTA of the first goes through all groups and its own group's requests, which 8192 requests in one group
// make 51 us (in 8 groups 14, in 64 or 512 12).

#include "gdr_kv8_split.cuh"

namespace gdr {
namespace {

// ------------------------------------------------------------------ plan
// A request is live if it has queries.  A group's lead is its first live request; what all live ones have
// in common are the first entries of their table rows up to the first in which one differs from the
// lead's, and no more than all of a request's queries see in whole pages.  A CTA compares one request's
// row (1000 rows of 4096 entries: all SMs read), then one takes the least of a group's.
constexpr int PT = 128;

struct PlanArgs {
    const int *table, *kv_len, *cu_q, *group;
    int *shared, *lead;
    int S, groups, W, page_log2;
};
__device__ __forceinline__ int queries_of(const PlanArgs &a, int s) { return a.cu_q ? a.cu_q[s + 1] - a.cu_q[s] : 1; }
// Whole pages that all queries of a live request see.
__device__ __forceinline__ int seen_pages(const PlanArgs &a, int s, int n) {
    const int64_t kv = min((int64_t)max(a.kv_len[s], 0), (int64_t)a.W << a.page_log2);
    return (int)(max(kv - n + 1, (int64_t)0) >> a.page_log2);
}
// The requests of group g, clamped.
__device__ __forceinline__ int2 requests_of(const PlanArgs &a, int g) {
    const int b = min(max(a.group[g], 0), a.S);
    return make_int2(b, min(max(a.group[g + 1], b), a.S));
}

// shared[s] = pages that request s has in common with its group's lead; -1 for a request without queries or
// alone with them, 0 for one in no group, which the second kernel does not come to.
__global__ void __launch_bounds__(PT) shared_rows_kernel(const PlanArgs a) {
    __shared__ int s_group, s_lead, s_live, s_limit, s_same;
    const int s = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) s_group = a.groups, s_lead = a.S, s_live = 0, s_limit = a.W;
    grid_dependency_wait();
    __syncthreads();
    for (int g = tid; g < a.groups; g += PT) {
        const int2 r = requests_of(a, g);
        if (s >= r.x && s < r.y) atomicMin(&s_group, g);
    }
    __syncthreads();
    int pages = s_group < a.groups ? -1 : 0;
    if (s_group < a.groups && queries_of(a, s) > 0) {
        const int2 r = requests_of(a, s_group);
        int lead = a.S, live = 0, limit = a.W;
        for (int i = r.x + tid; i < r.y; i += PT) {
            const int n = queries_of(a, i);
            if (n <= 0) continue;
            lead = min(lead, i);
            ++live;
            limit = min(limit, seen_pages(a, i, n));
        }
        atomicMin(&s_lead, lead);
        atomicAdd(&s_live, live);
        atomicMin(&s_limit, limit);
        __syncthreads();
        if (s_live > 1) {
            pages = s_limit;
            if (s != s_lead) {
                const int *mine = a.table + (int64_t)s * a.W, *theirs = a.table + (int64_t)s_lead * a.W;
                constexpr int U = 8;
                for (int c0 = 0; c0 < pages; c0 += U * PT) {
                    int x[U], y[U];
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int c = c0 + i * PT + tid;
                        x[i] = c < pages ? mine[c] : 0;
                        y[i] = c < pages ? theirs[c] : 0;
                    }
                    int differs = pages;
#pragma unroll
                    for (int i = U - 1; i >= 0; --i)
                        if (x[i] != y[i]) differs = c0 + i * PT + tid;
                    if (__syncthreads_or(differs < pages)) {
                        if (tid == 0) s_same = pages;
                        __syncthreads();
                        atomicMin(&s_same, differs);
                        __syncthreads();
                        pages = s_same;
                        break;
                    }
                }
            }
        }
    }
    if (tid == 0) a.shared[s] = pages;
    grid_launch_dependents();
}
// The least of a group's.
__global__ void __launch_bounds__(PT) shared_groups_kernel(const PlanArgs a) {
    __shared__ int s_pages, s_lead;
    const int g = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) s_pages = a.W, s_lead = a.S;
    grid_dependency_wait();
    __syncthreads();
    const int2 r = requests_of(a, g);
    int pages = a.W, lead = a.S;
    for (int i = r.x + tid; i < r.y; i += PT) {
        const int n = a.shared[i];
        if (n < 0) continue;
        pages = min(pages, n);
        lead = min(lead, i);
    }
    atomicMin(&s_pages, pages);
    atomicMin(&s_lead, lead);
    __syncthreads();
    const bool any = s_lead < a.S && s_pages > 0;
    for (int i = r.x + tid; i < r.y; i += PT) a.shared[i] = any && a.shared[i] >= 0 ? s_pages << a.page_log2 : 0;
    if (tid == 0) a.lead[g] = any ? s_lead : -1;
    grid_launch_dependents();
}

// ------------------------------------------------------------------ attention
size_t align32(size_t n) { return (n + 31) & ~(size_t)31; }
size_t pre_bytes(int total_q, int Hq, int D) { return align32((size_t)total_q * Hq * (D + 2) * sizeof(float)); }

// Common tokens from which on the first pass is worth its time, by the sizes that the host knows.
//
// What 128 common tokens of a cached head cost one SM, in us: the split kernel's blocks of 8 or 16 rows
// (measured: 128 decodes of 8 heads a cached head on 32 k common keys, from the L2 mostly, 502 us = 0.58 a
// block; fp32 1.0 and 1.6 at D = 128, 0.63 and 1.0 at 64), the tile kernel's copies, tile or pair of
// tiles (24 x 5 drafted tokens on 16 k 110 us = 1.3; 2.4 a pair).
// A pass of its own costs 15 us (16 decodes on 4096 common tokens 31 us against 21 in one), 19 where it
// takes pairs, the sums' way through memory, and the ends of items that are twice as many.
// Where the two are even, measured / by this rule, with 4 cached heads of 8 query heads: 8, 16, 32, 64 decodes
// 22 / 22, 9 / 10, 5.2 / 5.7, 2.9 / 2.9 thousand common tokens; 24 x 5 drafted 6 / 6; prompts of 64 or 300
// tokens: none up to 16 k / none, 20.  (2.4 a pair fits these; whole passes of many blocks took 2.6, above.)
// What the rule leaves out: lengths, so it does not see work that does not fill the SMs, nor a batch with
// groups on both sides of the bound.  75 decodes of 8 heads and one cached head in 6 groups of 10 to 21 k
// common tokens 46 us, gdr_kv8_attn 34; 18 x 2 to 5 drafted in groups of 0 to 31 k 99 and 36: some groups
// are below the bound, and the second pass's tile kernel takes 75 us for 8 requests' 16 k keys and 9 short items
// (without short ones, or in gdr_kv8_attn with 10 of them, the like takes 24; short items stand together, their
// ends read the first pass's sums in turn, and with so few units a CTA ends do not count in the division).
// Of 7543 drawn batches 3.1 % were more than a tenth slower than gdr_kv8_attn, 0.3 % more than half.
// (`rows` of one request or group on average, at most `most`; alike: all have that many, else the last
// block of each is half full; ends: what the ends of its items cost in units)
double keys_cost(int64_t most, double rows, bool alike, int D, Elem e, double *ends) {
    const double narrow = D == 64 ? 0.63 : 1.0;
    auto blocks = [&](int n) { return alike ? std::ceil(rows / n) : rows / n + 0.5; };
    *ends = sp::ITEM;
    if (e == Elem::F32) return most <= 8 ? narrow : 1.6 * narrow * blocks(16);
    if (most <= 16) return (most <= 8 ? 0.58 : 0.8) * narrow;
    *ends = most > 128 ? 3 : 8;
    return most <= 64 ? 1.3 : most <= 128 ? 1.7 : 2.4 * blocks(kKv8TileRows);
}
int least_worth(const KvSharedCall &c) {
    if (opt_shared_least() > 0) return opt_shared_least();
    const int64_t G = c.Hq / c.Hkv, most = c.max_q * G, gmost = c.max_group_q * G;
    const double requests = std::min(c.S, c.total_q), sms = sm_count();
    double ends, gends;
    const double one = keys_cost(most, c.total_q * G / requests, (int64_t)c.S * c.max_q == c.total_q, c.D, c.e, &ends);
    const double group = keys_cost(gmost, (double)c.total_q * G / c.groups, c.groups == 1, c.D, c.e, &gends);
    const double gain = requests * one - c.groups * group;
    if (gain <= 0) return 0x7fffffff;
    const double pass = (c.e == Elem::BF16 && gmost > 128 ? 19 : 15) + (double)c.total_q * c.Hq * (8 * c.D + 16) / 3e6 +
                        requests * c.Hkv * one * ends / sms;
    return (int)std::min(pass * sms / (gain * c.Hkv) * 128, 2147483647.0);
}

template <bool FIRST>
cudaError_t launch_pass(const KvSharedCall &c, float *pre_o, float2 *pre_ml, void *parts, cudaStream_t s) {
    const int max_q = FIRST ? c.max_group_q : c.max_q;
    const Shape sh = shape_of(max_q, c.Hq / c.Hkv, c.e);
    if (sh == Shape::TILE)
        return c.kv == Kv8::E4M3 ? launch_kv8_shared_e4m3(c, FIRST, pre_o, pre_ml, parts, s)
                                 : launch_kv8_shared_int8(c, FIRST, pre_o, pre_ml, parts, s);
    SharedArgs<FIRST> a = shared_args<FIRST>(c, pre_o, pre_ml);
    return launch_split_any(a, sh, c.k_cache, c.v_cache, c.D, c.e, c.kv, parts, (int64_t)max_q * a.G, s);
}

}  // namespace

cudaError_t launch_kv8_shared_plan(const int *table, const int *kv_len, const int *cu_q, const int *cu_group, int *shared,
                                   int *lead, int S, int groups, int W, int page, cudaStream_t s) {
    PlanArgs a{table, kv_len, cu_q, cu_group, shared, lead, S, groups, W, page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7};
    cudaError_t e = launch_after(shared_rows_kernel, dim3((unsigned)S), PT, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_after(shared_groups_kernel, dim3((unsigned)groups), PT, 0, s, a);
}

size_t kv8_shared_workspace_bytes(int max_q, int max_group_q, int total_q, int Hq, int Hkv, int D, Elem e) {
    const int G = Hq / Hkv;
    return pre_bytes(total_q, Hq, D) + std::max(shape_workspace_bytes(shape_of(max_group_q, G, e), D),
                                                shape_workspace_bytes(shape_of(max_q, G, e), D));
}

cudaError_t launch_kv8_shared(const KvSharedCall &call, void *ws, cudaStream_t s) {
    KvSharedCall c = call;
    c.least = least_worth(c);
    if ((int64_t)c.least > (int64_t)c.W * c.page)      // no request can have that many: one pass
        return launch_kv8_attn(c.q, c.q_stride, c.k_cache, c.v_cache, c.k_scale, c.v_scale, c.table, c.kv_len, c.cu_q,
                               c.scale, c.out, c.lse, c.S, c.max_q, c.total_q, c.Hq, c.Hkv, c.D, c.W, c.page, c.N, c.e,
                               c.kv, ws, s);
    float *pre_o = static_cast<float *>(ws);
    float2 *pre_ml = reinterpret_cast<float2 *>(pre_o + (size_t)c.total_q * c.Hq * c.D);
    void *parts = static_cast<uint8_t *>(ws) + pre_bytes(c.total_q, c.Hq, c.D);
    cudaError_t e = launch_pass<true>(c, pre_o, pre_ml, parts, s);
    if (e != cudaSuccess) return e;
    return launch_pass<false>(c, pre_o, pre_ml, parts, s);
}

cudaError_t take_kv8_shared_error_word(unsigned *value) { return take_attn_error_word(value); }

}  // namespace gdr
