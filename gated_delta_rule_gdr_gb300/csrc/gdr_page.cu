// gdr_page.cu -- block tables and slot maps of a paged cache, built on the device from the
// requests' lengths (gdr_page_plan).
//
// kv_s tokens cached, n_s new ones (n_s < 0: finished), pages of P tokens, W table columns:
//   old_s  = ceil(kv_s / P), or the pages held_s that its row has where that is more (tokens
//            were taken back), at most W
//   need_s = max(0, ceil((kv_s + n_s) / P) - old_s)
//   a request fits if kv_s + n_s <= W P and its tokens end within max_tokens; it is granted
//   if it fits and needs no page, or the fitting requests up to and including it need at
//   most `count` pages -- so the grant depends on the order of the requests alone
//   table[s][old_s + i] = ring[(head + sum_{r<s} need_r + i) mod N]
//   slot of token i     = table[s][(kv_s + i) / P] P + (kv_s + i) mod P, -1 where that entry is
//                         outside [0, N)
//   a finished request's old_s pages go behind the ring's last one and its length to 0;
//   entries of its row outside [0, N) are pages that are gone and stay out of the ring.
//
// Everything that a token's slot depends on beyond its own request is a prefix sum over
// requests, a few KB, so every CTA computes those sums for itself in shared memory (one
// read of the lengths from L2, three block scans) and then takes its share of tokens and
// new pages: one launch, no order between CTAs.  In place, and still without an order: tokens
// read only table entries below old_s and ring entries of this call's grants, the writes go
// to entries at or above old_s and behind the ring's end.  Released pages depend on what the
// table holds: one CTA, or one cluster where the table is large, counts and places them.
//
// Bound: the launch and the scans' latency (300 requests of one token, 9 of them finished, 7.0 us,
// 24 KB, 5.4 without a finished one; 60 prompts of some 250 k tokens together 7.5 us, 2.0 MB,
// of which the bytes are 0.3 us).

#include "gdr_internal.h"
#include "gdr_sm100.cuh"

#include <algorithm>

namespace gdr {
namespace {

constexpr int PT = 512;   // threads
// Entries of a finished request's row that a warp takes at a time: eight loads in flight a lane.
constexpr int CHUNK = 256;
// Table entries (S W) from which the launch has clusters of 8.  Eight CTAs that share the counting
// of released pages: 1500 requests, 30 % of them finished with up to 2048 pages each, 34 us; one
// CTA 106.  A launch with clusters takes 1.0 us more (9 of 300 finished, 256 pages each: 7.5 and
// 8.5 us), so small tables go without.
constexpr int64_t kClusterEntries = 1 << 19;

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
    const int *kv_len, *q_len, *held, *free_state;
    int *table, *ring, *kv_out, *cu_q, *slots, *positions, *granted, *held_out, *state_out;
    int S, W, page, N, max_tokens;
    int cluster;      // CTAs of the launch's clusters
};

__global__ void __launch_bounds__(PT) page_plan_kernel(const PlanArgs a) {
    extern __shared__ int sm[];
    int *s_cu = sm;                   // [S + 1] first token of a request, at most max_tokens
    int *s_need = sm + a.S + 1;       // [S + 1] pages granted before it
    int *s_fin = s_need + a.S + 1;    // [S] the finished requests that have pages, in order
    int *s_chunk = s_fin + a.S;       // [S + 1] chunks of their entries before each
    int *s_old = s_chunk + a.S + 1;   // [S] entries of each
    int *s_rel = s_old + a.S;         // [S + 1] pages that this CTA counted, then those released before it
    int *s_sum = s_rel + a.S + 1;     // [S] its pages
    __shared__ int64_t s_w64[PT / 32];
    __shared__ int s_w32[PT / 32];
    const int tid = threadIdx.x, S = a.S, P = a.page;
    const int room = a.W * P, shift = 31 - __clz(P);     // below 2^31; P is a power of two
    const int per = (S + PT - 1) / PT, s0 = min(S, tid * per), s1 = min(S, s0 + per);
    const int count = min(max(a.free_state[1], 0), a.N);
    const int head = (int)((unsigned)a.free_state[0] % (unsigned)a.N);
    auto kv_of = [&](int s) { return max(a.kv_len[s], 0); };
    auto pages_of = [&](int s, int kv) {        // that its row has
        const int least = (min(kv, room) + P - 1) >> shift;
        return a.held ? min(max(a.held[s], least), a.W) : least;
    };

    int64_t sum = 0, all;
    for (int s = s0; s < s1; ++s) sum += max(a.q_len[s], 0);
    int64_t at = block_exclusive<int64_t>(sum, s_w64, &all);
    int need = 0;
    int64_t fin = 0;                  // finished requests with pages << 32 | chunks of their entries
    for (int s = s0; s < s1; ++s) {
        const int kv = kv_of(s), n = a.q_len[s], old = pages_of(s, kv);
        s_cu[s] = (int)min(at, (int64_t)a.max_tokens);
        at += max(n, 0);
        // -1: does not fit
        int x = -1;
        if (n >= 0 && (int64_t)kv + n <= room && at <= a.max_tokens) x = max(((kv + n + P - 1) >> shift) - old, 0);
        s_need[s] = x;
        need += max(x, 0);
        if (n < 0 && old > 0) fin += (1ll << 32) + (old + CHUNK - 1) / CHUNK;
    }
    if (tid == 0) s_cu[S] = (int)min(all, (int64_t)a.max_tokens);
    int total_need;
    int64_t total_fin;
    int b_need = block_exclusive<int>(need, s_w32, &total_need);
    int64_t b_fin = block_exclusive<int64_t>(fin, s_w64, &total_fin);
    const int finished = (int)(total_fin >> 32), chunks = (int)total_fin;
    // a request that is not granted ends the grants: later ones need pages behind its own
    int last = 0;
    for (int s = s0; s < s1; ++s) {
        const int x = s_need[s];
        const bool ok = a.q_len[s] < 0 || x == 0 || (x > 0 && b_need + x <= count);
        const int upto = x > 0 ? b_need + x : b_need;
        s_need[s] = min(b_need, count);
        if (x > 0 && ok) last = upto;
        b_need = upto;
        const int kv = kv_of(s), n = a.q_len[s], old = pages_of(s, kv);
        if (n < 0 && old > 0) {
            s_fin[b_fin >> 32] = s;
            s_chunk[b_fin >> 32] = (int)b_fin;
            s_old[b_fin >> 32] = old;
            s_rel[b_fin >> 32] = 0;
            b_fin += (1ll << 32) + (old + CHUNK - 1) / CHUNK;
        }
        if (blockIdx.x == 0) {
            a.granted[s] = ok ? 1 : 0;
            a.kv_out[s] = n < 0 ? 0 : (ok ? kv + n : kv);
            a.cu_q[s] = s_cu[s];
            if (a.held) a.held_out[s] = n < 0 ? 0 : old + (ok ? max(x, 0) : 0);
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
        s_chunk[finished] = chunks;
        if (blockIdx.x == 0) a.cu_q[S] = s_cu[S];
    }
    __syncthreads();

    // A request's need and grant, from its own lengths and the prefix before it.
    auto granted_pages = [&](int s, int kv, int n, int old, int end) {   // -1: not granted
        if (n < 0 || (int64_t)kv + n > room || end > a.max_tokens) return -1;
        const int x = max(((kv + n + P - 1) >> shift) - old, 0);
        return x == 0 || s_need[s] + x <= taken ? x : -1;
    };
    const int stride = gridDim.x * PT, first = blockIdx.x * PT + tid;
    const int tokens = s_cu[S];
    for (int t = first; t < a.max_tokens; t += stride) {
        int slot = -1, pos = -1;
        if (t < tokens) {
            const int s = find_request(s_cu, S, t);
            const int kv = kv_of(s), n = a.q_len[s], old = pages_of(s, kv);
            // the end of the request's tokens: a saturated prefix means it does not fit
            const int64_t end = (int64_t)s_cu[s] + n;
            if (granted_pages(s, kv, n, old, (int)min(end, (int64_t)a.max_tokens + 1)) >= 0) {
                const int at = kv + (t - s_cu[s]), p = at >> shift;
                const int page = p < old ? a.table[(int64_t)s * a.W + p]
                                         : a.ring[((int64_t)head + s_need[s] + (p - old)) % a.N];
                if ((unsigned)page < (unsigned)a.N) {      // else a page that is gone: no place
                    pos = at;
                    slot = (page << shift) + (at & (P - 1));
                }
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
    for (int i = first; i < taken; i += stride) {
        const int s = find_request(s_need, S, i);
        const int old = pages_of(s, kv_of(s));
        a.table[(int64_t)s * a.W + old + (i - s_need[s])] = a.ring[((int64_t)head + i) % a.N];
    }

    // ---- the pages of finished requests.  A page's place in the ring depends on how many of the
    // entries before it are pages; the CTAs of one cluster count a share of the chunks each, add
    // up what the others counted, and write a share each.
    constexpr int NW = PT / 32, EACH = CHUNK / 32;
    if ((int)blockIdx.x >= a.cluster) return;
    const int warp = tid >> 5, lane = tid & 31, c0 = blockIdx.x * NW + warp, step = a.cluster * NW;
    auto there = [&](int page) { return (unsigned)page < (unsigned)a.N; };
    auto load_chunk = [&](int c, int &f, int (&page)[EACH]) {   // of request f; -1 past its row
        f = find_request(s_chunk, finished, c);
        const int i0 = (c - s_chunk[f]) * CHUNK + lane, old = s_old[f];
        const int *row = a.table + (int64_t)s_fin[f] * a.W + i0;
#pragma unroll
        for (int j = 0; j < EACH; ++j) page[j] = i0 + 32 * j < old ? row[32 * j] : -1;
    };
    int keep[EACH], keep_f = 0, total_rel = 0;        // a warp's first chunk stays in registers
    if (finished > 0) {
        auto add = [&](int f, const int (&page)[EACH]) {
            int n = 0;
#pragma unroll
            for (int j = 0; j < EACH; ++j) n += there(page[j]);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) atomicAdd(&s_rel[f], n);
        };
        if (c0 < chunks) load_chunk(c0, keep_f, keep), add(keep_f, keep);
        int c = c0 + step, f[4], page[4][EACH];
        for (; c + 3 * step < chunks; c += 4 * step) {   // four at once: the loads of many
#pragma unroll
            for (int u = 0; u < 4; ++u) load_chunk(c + u * step, f[u], page[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) add(f[u], page[u]);
        }
        for (; c < chunks; c += step) load_chunk(c, f[0], page[0]), add(f[0], page[0]);
        const int each = (finished + PT - 1) / PT, f0 = min(finished, tid * each), f1 = min(finished, f0 + each);
        int n = 0;
        if (a.cluster > 1) {
            sm100::cluster_sync();
            for (int g = f0; g < f1; ++g) {
                int sum = 0;
                for (int r = 0; r < a.cluster; ++r)
                    sum += (int)sm100::ld_cluster_u32(sm100::cluster_map(sm100::smem_u32(s_rel + g), r));
                s_sum[g] = sum;
                n += sum;
            }
            sm100::cluster_sync();        // nobody writes its counts, or leaves, while others read them
        } else {
            __syncthreads();
            for (int g = f0; g < f1; ++g) n += s_sum[g] = s_rel[g];
        }
        int b = block_exclusive<int>(n, s_w32, &total_rel);
        for (int g = f0; g < f1; ++g) {
            s_rel[g] = b;
            b += s_sum[g];
        }
        if (tid == 0) s_rel[finished] = total_rel;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.state_out[0] = (int)(((unsigned)head + (unsigned)taken) % (unsigned)a.N);
        a.state_out[1] = (int)min((int64_t)count - taken + total_rel, (int64_t)a.N);
    }
    for (int c = c0; c < chunks; c += step) {
        if (c != c0) load_chunk(c, keep_f, keep);
        const int f = keep_f, i0 = (c - s_chunk[f]) * CHUNK, old = s_old[f];
        // num_pages is below 2^27 and the entries of all rows below 2^31
        const unsigned N = a.N, to = ((unsigned)head + (unsigned)count + (unsigned)s_rel[f] + (unsigned)i0) % N;
        if (s_sum[f] == old) {                               // every entry is a page
            unsigned at = (to + lane) % N;
#pragma unroll
            for (int j = 0; j < EACH; ++j) {
                if (i0 + 32 * j + lane < old) a.ring[at] = keep[j];
                at += 32;                    // N may be less than 32
                at = at < N ? at : at - N < N ? at - N : at % N;
            }
        } else if (i0 == 0) {                                // some are gone: one warp the whole row
            const int *row = a.table + (int64_t)s_fin[f] * a.W;
            for (unsigned i = lane, before = 0; i - lane < (unsigned)old; i += 32) {
                const int page = i < (unsigned)old ? row[i] : -1;
                const unsigned m = __ballot_sync(0xffffffffu, there(page));
                if (there(page)) a.ring[(to + before + __popc(m & ((1u << lane) - 1))) % N] = page;
                before += __popc(m);
            }
        }
    }
}

}  // namespace

size_t page_plan_smem(int S) { return ((size_t)7 * S + 4) * sizeof(int); }

cudaError_t launch_page_plan(const int *kv_len, const int *q_len, const int *held, int *table, int *ring,
                             const int *free_state, int *kv_out, int *cu_q, int *slots, int *positions,
                             int *granted, int *held_out, int *state_out, int S, int W, int page, int N, int max_tokens,
                             cudaStream_t s) {
    // about four tokens or requests a thread: the scans repeat in every CTA, so more CTAs cost nothing
    const int64_t items = (int64_t)max_tokens + 16ll * S;
    int64_t blocks = std::min(std::max((items + 4 * PT - 1) / (4 * PT), (int64_t)1), (int64_t)304);
    const int cluster = (int64_t)S * W >= kClusterEntries ? 8 : 1;
    blocks = (blocks + cluster - 1) / cluster * cluster;
    const PlanArgs a{kv_len, q_len, held, free_state, table, ring, kv_out, cu_q, slots, positions, granted,
                     held_out, state_out, S, W, page, N, max_tokens, cluster};
    const size_t smem = page_plan_smem(S);
    if (smem > 48 * 1024) {
        // the limit is the kernel's, on every thread: always what the largest batch needs
        cudaError_t e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)page_plan_smem(kMaxRequests));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(PT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, page_plan_kernel, a);
}

}  // namespace gdr
