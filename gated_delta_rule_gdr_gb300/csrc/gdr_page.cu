// gdr_page.cu -- block tables and slot maps of a paged cache, built on the device from the
// requests' lengths (gdr_page_plan).
//
// kv_s tokens cached, n_s new ones (n_s < 0: finished), pages of P tokens, W table columns:
//   old_s  = ceil(kv_s / P),  need_s = ceil((kv_s + n_s) / P) - old_s
//   a request fits if kv_s + n_s <= W P and its tokens end within max_tokens; it is granted
//   if it fits and needs no page, or the fitting requests up to and including it need at
//   most `count` pages -- so the grant depends on the order of the requests alone
//   table[s][old_s + i] = ring[(head + sum_{r<s} need_r + i) mod N]
//   slot of token i     = table[s][(kv_s + i) / P] P + (kv_s + i) mod P
//   a finished request's old_s pages go behind the ring's last one and its length to 0.
//
// Everything that a token's slot depends on beyond its own request is a prefix sum over
// requests, a few KB, so every CTA computes those sums for itself in shared memory (one
// read of the lengths from L2, three block scans) and then takes its share of tokens, new
// pages and released pages: one launch, no order between CTAs.  In place, and still
// without an order: tokens read only table entries below old_s and ring entries of this
// call's grants, the writes go to entries at or above old_s and behind the ring's end.
//
// Bound: the launch and the scans' latency (300 requests of one token 6.6 us, 24 KB; 60 prompts
// of some 250 k tokens together 8.0 us, 2.0 MB, of which the bytes are 0.3 us).

#include "gdr_internal.h"

namespace gdr {
namespace {

constexpr int PT = 512;   // threads

// Exclusive block-wide prefix sum of one value per thread; *total gets the sum.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T *s_warp, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < PT / 32; ++w) {
        const T x = s_warp[w];
        if (w < warp) before += x;
        all += x;
    }
    *total = all;
    return before + incl - v;
}

// The request of item i: the last s with prefix[s] <= i (prefix[S] > i).
__device__ __forceinline__ int find_request(const int *prefix, int S, int i) {
    int lo = 0, hi = S;   // prefix[lo] <= i < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

struct PlanArgs {
    const int *kv_len, *q_len, *free_state;
    int *table, *ring, *kv_out, *cu_q, *slots, *positions, *granted, *state_out;
    int S, W, page, N, max_tokens;
};

__global__ void __launch_bounds__(PT) page_plan_kernel(const PlanArgs a) {
    extern __shared__ int sm[];
    int *s_cu = sm;                   // [S + 1] first token of a request, at most max_tokens
    int *s_need = sm + a.S + 1;       // [S + 1] pages granted before it
    int *s_rel = s_need + a.S + 1;    // [S + 1] pages released before it
    __shared__ int64_t s_w64[PT / 32];
    __shared__ int s_w32[PT / 32];
    const int tid = threadIdx.x, S = a.S, P = a.page;
    const int64_t room = (int64_t)a.W * P;
    const int per = (S + PT - 1) / PT, s0 = min(S, tid * per), s1 = min(S, s0 + per);
    const int count = min(max(a.free_state[1], 0), a.N);
    const int head = (int)((unsigned)a.free_state[0] % (unsigned)a.N);
    auto kv_of = [&](int s) { return (int)min((int64_t)max(a.kv_len[s], 0), room); };

    int64_t sum = 0, all;
    for (int s = s0; s < s1; ++s) sum += max(a.q_len[s], 0);
    int64_t at = block_exclusive<int64_t>(sum, s_w64, &all);
    int need = 0, rel = 0;
    for (int s = s0; s < s1; ++s) {
        const int kv = kv_of(s), n = a.q_len[s], old = (kv + P - 1) / P;
        s_cu[s] = (int)min(at, (int64_t)a.max_tokens);
        at += max(n, 0);
        // -1: does not fit
        int x = -1;
        if (n >= 0 && (int64_t)kv + n <= room && at <= a.max_tokens) x = (kv + n + P - 1) / P - old;
        s_need[s] = x;
        s_rel[s] = n < 0 ? old : 0;
        need += max(x, 0);
        rel += s_rel[s];
    }
    if (tid == 0) s_cu[S] = (int)min(all, (int64_t)a.max_tokens);
    int total_need, total_rel;
    int b_need = block_exclusive<int>(need, s_w32, &total_need);
    int b_rel = block_exclusive<int>(rel, s_w32, &total_rel);
    // a request that is not granted ends the grants: later ones need pages behind its own
    int last = 0;
    for (int s = s0; s < s1; ++s) {
        const int x = s_need[s];
        const bool ok = a.q_len[s] < 0 || x == 0 || (x > 0 && b_need + x <= count);
        const int upto = x > 0 ? b_need + x : b_need;
        s_need[s] = min(b_need, count);
        if (x > 0 && ok) last = upto;
        b_need = upto;
        const int r = s_rel[s];
        s_rel[s] = b_rel;
        b_rel += r;
        if (blockIdx.x == 0) {
            const int kv = kv_of(s), n = a.q_len[s];
            a.granted[s] = ok ? 1 : 0;
            a.kv_out[s] = n < 0 ? 0 : (ok ? kv + n : kv);
            a.cu_q[s] = s_cu[s];
        }
    }
    // pages granted in all: the largest prefix that a granted request reaches
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, off));
    __syncthreads();
    if ((tid & 31) == 0) s_w32[tid >> 5] = last;
    __syncthreads();
    int taken = 0;
#pragma unroll
    for (int w = 0; w < PT / 32; ++w) taken = max(taken, s_w32[w]);
    if (tid == 0) {
        s_need[S] = total_need;
        s_rel[S] = total_rel;
        if (blockIdx.x == 0) {
            a.cu_q[S] = s_cu[S];
            a.state_out[0] = (int)(((int64_t)head + taken) % a.N);
            a.state_out[1] = (int)min((int64_t)count - taken + total_rel, (int64_t)a.N);
        }
    }
    __syncthreads();

    // A request's need and grant, from its own lengths and the prefix before it.
    auto granted_pages = [&](int s, int kv, int n, int end) {   // -1: not granted
        if (n < 0 || (int64_t)kv + n > room || end > a.max_tokens) return -1;
        const int x = (kv + n + P - 1) / P - (kv + P - 1) / P;
        return x == 0 || s_need[s] + x <= taken ? x : -1;
    };
    const int stride = gridDim.x * PT, first = blockIdx.x * PT + tid;
    const int tokens = s_cu[S];
    for (int t = first; t < a.max_tokens; t += stride) {
        int slot = -1, pos = -1;
        if (t < tokens) {
            const int s = find_request(s_cu, S, t);
            const int kv = kv_of(s), n = a.q_len[s], old = (kv + P - 1) / P;
            // the end of the request's tokens: a saturated prefix means it does not fit
            const int64_t end = (int64_t)s_cu[s] + n;
            if (granted_pages(s, kv, n, (int)min(end, (int64_t)a.max_tokens + 1)) >= 0) {
                pos = kv + (t - s_cu[s]);
                const int p = pos / P;
                const int page = p < old ? a.table[(int64_t)s * a.W + p]
                                         : a.ring[((int64_t)head + s_need[s] + (p - old)) % a.N];
                slot = page * P + (pos - p * P);
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    for (int i = first; i < taken; i += stride) {
        const int s = find_request(s_need, S, i);
        const int old = (kv_of(s) + P - 1) / P;
        a.table[(int64_t)s * a.W + old + (i - s_need[s])] = a.ring[((int64_t)head + i) % a.N];
    }
    for (int i = first; i < total_rel; i += stride) {
        const int s = find_request(s_rel, S, i);
        a.ring[((int64_t)head + count + i) % a.N] = a.table[(int64_t)s * a.W + (i - s_rel[s])];
    }
}

}  // namespace

size_t page_plan_smem(int S) { return (size_t)3 * (S + 1) * sizeof(int); }

cudaError_t launch_page_plan(const int *kv_len, const int *q_len, int *table, int *ring,
                             const int *free_state, int *kv_out, int *cu_q, int *slots, int *positions,
                             int *granted, int *state_out, int S, int W, int page, int N, int max_tokens,
                             cudaStream_t s) {
    const PlanArgs a{kv_len, q_len, free_state, table, ring, kv_out, cu_q, slots, positions, granted,
                     state_out, S, W, page, N, max_tokens};
    const size_t smem = page_plan_smem(S);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    // about four tokens or requests a thread: the scans repeat in every CTA, so more CTAs cost nothing
    const int64_t items = (int64_t)max_tokens + 16ll * S;
    const int64_t blocks = (items + 4 * PT - 1) / (4 * PT);
    page_plan_kernel<<<(unsigned)(blocks < 1 ? 1 : (blocks > 304 ? 304 : blocks)), PT, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gdr
