// Page bookkeeping of a paged cache, on the device: the step a scheduler makes between two
// model steps (free, fork, reserve with copy-on-write) and the compaction of a pool.
//
// State: page_table[s][i] = the page holding tokens i * page_tokens ... of sequence s (-1:
// none), page_ref[p] = table entries equal to p (0: free).  Sequences with a common prefix
// share its pages; a page is only written while one sequence has it, so before an append
// every page in the appended range that is missing or shared is replaced by a free one,
// its contents copied when it already holds tokens of the sequence.
//
// Every decision is a function of the state alone (free pages are taken lowest first, in
// the order of (sequence, place)), so results do not depend on timing.  The bookkeeping is
// a few thousand integers with many dependent steps: one CTA of 1,024 threads, phases
// separated by barriers, one round trip to memory per phase.  The page contents are moved
// by a second kernel, launched as a programmatic dependent, that reads the list the first
// one left: 16 KiB per CTA step, every pool in one launch.

#include <climits>

#include "qsa_internal.cuh"

namespace qsa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = kMoveThreads * 16 * 4;   // bytes a CTA moves per step

struct PagesHead {
    int n_moves;
    int n_live;
    int pad[62];
};

// Exclusive sum over the block and its total; every thread calls it.
__device__ __forceinline__ int block_scan(int v, int* total)
{
    __shared__ int s_sum[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int t = s_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
    }
    *total = __shfl_sync(0xffffffffu, t, 31);
    const int before = warp > 0 ? __shfl_sync(0xffffffffu, t, warp - 1) : 0;
    __syncthreads();   // s_sum may be written again
    return before + x - v;
}

// What a place of a table needs before an append: 0 nothing, 1 a page, 2 a page with the
// old one's contents.
__device__ __forceinline__ int place_needs(int e, int64_t n_pages, const int32_t* ref, bool holds_tokens)
{
    if (e < 0 || e >= n_pages) return 1;
    return __ldcg(ref + e) > 1 ? (holds_tokens ? 2 : 1) : 0;
}

}  // namespace

struct PagesWork {
    PagesHead* head;
    int32_t* claim;    // [batch] first fork of a target
    int32_t* mark;     // [batch] target that is also a source, or holds pages
    int32_t* count;    // [batch] pages a sequence needs, then the rank of its first
    int32_t* free_id;  // [n_pages] free pages, lowest first
    int32_t* drop;     // [n_pages] page a request leaves, or -1
    int32_t* remap;    // [n_pages] new id of a page (compaction)
    int2* moves;       // [max(batch, n_pages / 2 + 1)] (from, to)
};

__global__ void __launch_bounds__(kPlanThreads)
k_pages_update(int32_t* table, int32_t* ref, int batch, int table_ld, int page_tokens, int n_pages, int64_t kv_capacity,
               const int32_t* __restrict__ free_seq, int n_free, const int32_t* __restrict__ fork_src,
               const int32_t* __restrict__ fork_dst, int n_fork, const int32_t* __restrict__ len_before,
               const int32_t* __restrict__ len_after, PagesWork W, unsigned* status)
{
    __shared__ int s_moves;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();   // the mover waits for this kernel's end before it reads anything

    // ---- free: a place is emptied by whoever swaps its entry out, so a sequence may be named twice ----
    for (int64_t k = tid; k < (int64_t)n_free * table_ld; k += kPlanThreads) {
        const int s = __ldg(free_seq + k / table_ld);
        if (s < 0 || s >= batch) {
            set_status(status, QSA_DEV_BAD_SEQ);
            continue;
        }
        const int e = atomicExch(table + (int64_t)s * table_ld + k % table_ld, -1);
        if (e >= 0 && e < n_pages) atomicSub(ref + e, 1);
    }
    if (tid == 0) s_moves = 0;

    // ---- fork: a target counts once (its first fork), holds nothing and is nobody's source ----
    auto fork_ok = [&](int f, int& src, int& dst) {
        src = __ldg(fork_src + f);
        dst = __ldg(fork_dst + f);
        return src >= 0 && src < batch && dst >= 0 && dst < batch && src != dst;
    };
    if (n_fork > 0) {
        int src, dst;
        for (int f = tid; f < n_fork; f += kPlanThreads)
            if (fork_ok(f, src, dst)) {
                W.claim[dst] = INT_MAX;
                W.mark[dst] = 0;
            }
        __syncthreads();
        for (int f = tid; f < n_fork; f += kPlanThreads)
            if (fork_ok(f, src, dst)) {
                atomicMin(W.claim + dst, f);
                W.mark[src] = 1;
            }
        for (int64_t k = tid; k < (int64_t)n_fork * table_ld; k += kPlanThreads)
            if (fork_ok((int)(k / table_ld), src, dst) && __ldcg(table + (int64_t)dst * table_ld + k % table_ld) >= 0)
                W.mark[dst] = 1;
        __syncthreads();
        for (int64_t k = tid; k < (int64_t)n_fork * table_ld; k += kPlanThreads) {
            const int f = (int)(k / table_ld);
            if (!fork_ok(f, src, dst) || __ldcg(W.claim + dst) != f || __ldcg(W.mark + dst) != 0) {
                set_status(status, QSA_DEV_BAD_SEQ);
                continue;
            }
            int e = __ldcg(table + (int64_t)src * table_ld + k % table_ld);
            if (e >= n_pages) {
                set_status(status, QSA_DEV_BAD_PAGE);
                e = -1;
            }
            table[(int64_t)dst * table_ld + k % table_ld] = e;
            if (e >= 0) atomicAdd(ref + e, 1);
        }
    }
    __syncthreads();

    // ---- reserve, first pass: how many pages each sequence needs (a warp per sequence) ----
    auto range = [&](int s, int& lo, int& hi, int& lb) {
        lb = __ldg(len_before + s);
        const int la = __ldg(len_after + s);
        lo = hi = 0;
        if (lb < 0 || la < lb || la > kv_capacity) return false;
        if (la > lb) {
            lo = lb / page_tokens;
            hi = (la - 1) / page_tokens + 1;
        }
        return true;
    };
    for (int s = warp; s < batch; s += kPlanThreads / 32) {
        int lo, hi, lb, n = 0;
        if (!range(s, lo, hi, lb) && lane == 0) set_status(status, QSA_DEV_BAD_LEN);
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const int i = i0 + lane;
            const bool need =
                i < hi && place_needs(__ldcg(table + (int64_t)s * table_ld + i), n_pages, ref, (int64_t)i * page_tokens < lb);
            n += __popc(__ballot_sync(0xffffffffu, need));
        }
        if (lane == 0) W.count[s] = n;
    }
    __syncthreads();
    int wanted = 0;
    for (int s0 = 0; s0 < batch; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int total;
        const int at = block_scan(s < batch ? W.count[s] : 0, &total);
        if (s < batch) W.count[s] = wanted + at;
        wanted += total;   // at most the table's entries
    }

    // ---- the lowest free pages ----
    int found = 0;
    for (int p0 = 0; p0 < n_pages && found < wanted; p0 += kPlanThreads * 8) {
        unsigned mask = 0;
        const int base = p0 + tid * 8;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (base + u < n_pages && __ldcg(ref + base + u) == 0) mask |= 1u << u;
        int total;
        int at = found + block_scan(__popc(mask), &total);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (mask >> u & 1u) {
                if (at < wanted) W.free_id[at] = base + u;
                ++at;
            }
        found += total;
    }
    found = min(found, wanted);
    if (found < wanted && tid == 0) set_status(status, QSA_DEV_BAD_PAGE);
    __syncthreads();

    // ---- second pass: the same decisions (counts of the pages looked at have not changed: a page
    // taken here had none), requests served in order while there are pages ----
    for (int s = warp; s < batch && found > 0; s += kPlanThreads / 32) {
        int lo, hi, lb, at = W.count[s];
        range(s, lo, hi, lb);
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const int i = i0 + lane;
            int32_t* place = table + (int64_t)s * table_ld + i;
            const int e = i < hi ? __ldcg(place) : 0;
            const int needs = i < hi ? place_needs(e, n_pages, ref, (int64_t)i * page_tokens < lb) : 0;
            const unsigned who = __ballot_sync(0xffffffffu, needs != 0);
            const int rank = at + __popc(who & ((1u << lane) - 1u));
            at += __popc(who);
            if (needs == 0 || rank >= found) continue;
            const int to = W.free_id[rank];
            W.drop[rank] = e >= 0 && e < n_pages ? e : -1;
            if (needs == 2) W.moves[atomicAdd(&s_moves, 1)] = make_int2(e, to);
            *place = to;
        }
    }
    __syncthreads();
    // ---- counts: pages taken have one holder, pages left one less ----
    for (int r = tid; r < found; r += kPlanThreads) {
        ref[W.free_id[r]] = 1;
        if (W.drop[r] >= 0) atomicSub(ref + W.drop[r], 1);
    }
    if (tid == 0) W.head->n_moves = s_moves;
}

__global__ void __launch_bounds__(kPlanThreads)
k_pages_compact(int32_t* ref, int n_pages, PagesWork W, int32_t* n_live_out)
{
    const int tid = threadIdx.x;
    griddep_launch_dependents();
    int n_live = 0;
    for (int p0 = 0; p0 < n_pages; p0 += kPlanThreads * 8) {
        int n = 0;
        const int base = p0 + tid * 8;
#pragma unroll
        for (int u = 0; u < 8; ++u) n += base + u < n_pages && __ldcg(ref + base + u) > 0;
        int total;
        block_scan(n, &total);
        n_live += total;
    }
    // k-th free id below n_live takes the k-th live id from n_live on: as many of one as of the other
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < n_pages; p0 += kPlanThreads * 8) {
        unsigned mask = 0;
        const int base = p0 + tid * 8;
        int n_hole = 0, n_move = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int p = base + u;
            if (p >= n_pages) continue;
            const bool live = __ldcg(ref + p) > 0;
            if (p < n_live ? !live : live) mask |= 1u << u;
            if (p >= n_live && !live) W.remap[p] = -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (mask >> u & 1u) (base + u < n_live ? n_hole : n_move)++;
        int th, tm;
        int ah = holes + block_scan(n_hole, &th), am = movers + block_scan(n_move, &tm);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (mask >> u & 1u) {
                if (base + u < n_live) W.moves[ah++].y = base + u;
                else W.moves[am++].x = base + u;
            }
        holes += th;
        movers += tm;
    }
    __syncthreads();
    for (int k = tid; k < holes; k += kPlanThreads) {
        const int2 mv = W.moves[k];
        W.remap[mv.x] = mv.y;
        ref[mv.y] = ref[mv.x];
        ref[mv.x] = 0;
    }
    if (tid == 0) {
        W.head->n_moves = holes;
        W.head->n_live = n_live;
        *n_live_out = n_live;
    }
}

// Moves the listed pages of every pool; with `table` != null also renames its entries.
__global__ void __launch_bounds__(kMoveThreads)
k_pages_move(const __grid_constant__ qsa_page_pools P, PagesWork W, int32_t* table, int64_t n_entries)
{
    griddep_wait();
    const int tid = threadIdx.x;
    if (table) {
        const int n_live = __ldcg(&W.head->n_live);
        for (int64_t k = (int64_t)blockIdx.x * kMoveThreads + tid; k < n_entries; k += (int64_t)gridDim.x * kMoveThreads) {
            const int e = table[k];
            if (e >= n_live && e < P.n_pages) table[k] = __ldcg(W.remap + e);
        }
    }
    const int n_moves = __ldcg(&W.head->n_moves);
    int64_t first = 0;   // steps of the pools before this one
    for (int i = 0; i < P.n_pools; ++i) {
        const int64_t bytes = P.page_bytes[i];
        const int per_page = (int)((bytes + kMoveBytes - 1) / kMoveBytes);
        const int64_t steps = (int64_t)n_moves * per_page;
        // this CTA's steps of the grid-strided sequence that fall into pool i
        int64_t k = (int64_t)blockIdx.x - first % gridDim.x;
        if (k < 0) k += gridDim.x;
        for (; k < steps; k += gridDim.x) {
            const int2 mv = __ldcg(W.moves + k / per_page);
            const int64_t at = (int64_t)(k % per_page) * kMoveBytes + tid * 16;
            const char* src = (const char*)P.pool[i] + mv.x * bytes + at;
            char* dst = (char*)P.pool[i] + mv.y * bytes + at;
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (at + u * (kMoveThreads * 16) < bytes) v[u] = __ldcs((const uint4*)(src + u * (kMoveThreads * 16)));
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (at + u * (kMoveThreads * 16) < bytes) __stcs((uint4*)(dst + u * (kMoveThreads * 16)), v[u]);
        }
        first += steps;
    }
}

// ---------------------------------------------------------------- host side

namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Scratch behind the region every call keeps zeroed (status word, split counters).
size_t pages_layout(int batch, int64_t n_pages, char* ws, PagesWork* w)
{
    size_t off = up256(256 + attn_counter_bytes());
    auto take = [&](size_t bytes) {
        char* p = ws + off;
        off += up256(bytes);
        return p;
    };
    const int64_t moves = batch > n_pages / 2 + 1 ? batch : n_pages / 2 + 1;
    PagesWork t;
    t.head = (PagesHead*)take(sizeof(PagesHead));
    t.claim = (int32_t*)take((size_t)batch * 4);
    t.mark = (int32_t*)take((size_t)batch * 4);
    t.count = (int32_t*)take((size_t)batch * 4);
    t.free_id = (int32_t*)take((size_t)n_pages * 4);
    t.drop = (int32_t*)take((size_t)n_pages * 4);
    t.remap = (int32_t*)take((size_t)n_pages * 4);
    t.moves = (int2*)take((size_t)moves * 8);
    if (w) *w = t;
    return off;
}

}  // namespace

size_t pages_workspace_bytes(const qsa_dims& d, int64_t n_pages) { return pages_layout(d.batch, n_pages, nullptr, nullptr); }

static cudaError_t launch_move(const qsa_page_pools& p, const PagesWork& w, int32_t* table, int64_t n_entries,
                               cudaStream_t st)
{
    // enough CTAs to keep every SM's loads in flight; they stride over the list
    return launch_k(k_pages_move, dim3(148 * 8), dim3(kMoveThreads), 0, st, true, p, w, table, n_entries);
}

cudaError_t launch_pages_update(const qsa_dims& d, const qsa_page_pools& p, int32_t* page_table, int32_t* page_ref,
                                const int32_t* free_seq, int32_t n_free, const int32_t* fork_src,
                                const int32_t* fork_dst, int32_t n_fork, const int32_t* len_before,
                                const int32_t* len_after, char* ws, cudaStream_t st)
{
    PagesWork w;
    pages_layout(d.batch, p.n_pages, ws, &w);
    const int ld = (int)(d.kv_capacity / p.page_tokens);
    cudaError_t e = launch_k(k_pages_update, dim3(1), dim3(kPlanThreads), 0, st, false, page_table, page_ref, d.batch, ld,
                             p.page_tokens, (int)p.n_pages, d.kv_capacity, free_seq, n_free, fork_src, fork_dst, n_fork,
                             len_before, len_after, w, (unsigned*)ws);
    if (e != cudaSuccess || p.n_pools == 0) return e;
    return launch_move(p, w, nullptr, 0, st);
}

cudaError_t launch_pages_compact(const qsa_dims& d, const qsa_page_pools& p, int32_t* page_table, int32_t* page_ref,
                                 int32_t* n_live, char* ws, cudaStream_t st)
{
    PagesWork w;
    pages_layout(d.batch, p.n_pages, ws, &w);
    cudaError_t e = launch_k(k_pages_compact, dim3(1), dim3(kPlanThreads), 0, st, false, page_ref, (int)p.n_pages, w, n_live);
    if (e != cudaSuccess) return e;
    return launch_move(p, w, page_table, (int64_t)d.batch * (d.kv_capacity / p.page_tokens), st);
}

}  // namespace qsa
