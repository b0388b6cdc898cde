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
// a few thousand integers with about ten dependent round trips to memory: one CTA of 1,024
// threads, phases separated by barriers, the loads of a phase all under way at once.  The
// page contents are moved by a second kernel, launched as a programmatic dependent, that
// reads the list the first one left: 16 KiB per CTA step, every pool in one launch.
//
// Measured: a step of 128 sequences (32 freed, 16 forked, 33 tokens each) 21 us of bookkeeping
// and 5.6 us of copies with cold caches, 23 us in all otherwise; compaction of 2,048 pages of
// 147 KB (604 MB read and written) 92 us of copies, 6.5 TB/s, and 8 us of bookkeeping.

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

}  // namespace

struct PagesWork {
    PagesHead* head;
    int32_t* claim;     // [batch] first fork of a target
    int32_t* mark;      // [batch] target that is also a source, or holds pages
    int32_t* free_id;   // [n_pages] free pages, lowest first
    uint32_t* place;    // [n_pages] requests in order: place in the table, bit 31: with the old page's contents
    int32_t* drop;      // [n_pages] page a request leaves, or -1
    int32_t* remap;     // [n_pages] new id of a page (compaction)
    int2* moves;        // [max(batch, n_pages / 2 + 1)] (from, to)
};

namespace {

// Entries of `n` rows of a table, four at a time per thread: load(row, column) of the four is
// under way before use(row, column, value) of the first.
template <typename Load, typename Use>
__device__ __forceinline__ void for_entries(uint32_t n, uint32_t ld, Load load, Use use)
{
    const uint32_t total = n * ld;
    for (uint32_t k0 = threadIdx.x; k0 < total; k0 += 4 * kPlanThreads) {
        int v[4];
        uint32_t row[4], col[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t k = k0 + u * kPlanThreads;
            row[u] = k / ld;
            col[u] = k - row[u] * ld;
            v[u] = k < total ? load(row[u], col[u]) : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k0 + u * kPlanThreads < total) use(row[u], col[u], v[u]);
    }
}

// Eight counts from `base` on (a multiple of 8) as a mask of those that are 0; pages past the
// end count as taken.
__device__ __forceinline__ unsigned free_mask(const int32_t* ref, int base, int n_pages)
{
    int r[8];
    if (base + 8 <= n_pages) {
        const int4 a = __ldcg(reinterpret_cast<const int4*>(ref + base)), b = __ldcg(reinterpret_cast<const int4*>(ref + base) + 1);
        r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w, r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) r[u] = base + u < n_pages ? __ldcg(ref + base + u) : 1;
    }
    unsigned m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) m |= (unsigned)(r[u] <= 0) << u;
    return m;
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads)
k_pages_update(int32_t* table, int32_t* ref, int batch, int table_ld, int page_tokens, int n_pages, int64_t kv_capacity,
               const int32_t* __restrict__ free_seq, int n_free, const int32_t* __restrict__ fork_src,
               const int32_t* __restrict__ fork_dst, int n_fork, const int32_t* __restrict__ len_before,
               const int32_t* __restrict__ len_after, PagesWork W, unsigned* status)
{
    __shared__ int s_moves;
    __shared__ int s_at[kPlanThreads], s_lo[kPlanThreads], s_lb[kPlanThreads];
    const int tid = threadIdx.x;
    // before any wait, against the rule at launch_k: this kernel is itself launched without a programmatic
    // dependency, so all that is older has ended, and the mover waits for its end before it reads anything
    griddep_launch_dependents();
    if (tid == 0) s_moves = 0;

    // ---- free: a place is emptied by whoever swaps its entry out, so a sequence may be named twice ----
    for_entries(
        n_free, table_ld,
        [&](uint32_t f, uint32_t c) {
            const int s = __ldg(free_seq + f);
            if (s < 0 || s >= batch) {
                set_status(status, QSA_DEV_BAD_SEQ);
                return -1;
            }
            return atomicExch(table + (int64_t)s * table_ld + c, -1);
        },
        [&](uint32_t, uint32_t, int e) {
            if (e >= n_pages) set_status(status, QSA_DEV_BAD_PAGE);
            else if (e >= 0) atomicSub(ref + e, 1);
        });

    // ---- fork: a target counts once (its first fork), holds nothing and is nobody's source ----
    if (n_fork > 0) {
        auto named = [&](int f, int& src, int& dst) {
            src = __ldg(fork_src + f);
            dst = __ldg(fork_dst + f);
            return src >= 0 && src < batch && dst >= 0 && dst < batch && src != dst;
        };
        int src, dst;
        for (int f = tid; f < n_fork; f += kPlanThreads)
            if (named(f, src, dst)) {
                W.claim[dst] = INT_MAX;
                W.mark[dst] = 0;
            } else {
                set_status(status, QSA_DEV_BAD_SEQ);
            }
        __syncthreads();   // the freed places are empty, too
        for (int f = tid; f < n_fork; f += kPlanThreads)
            if (named(f, src, dst)) {
                atomicMin(W.claim + dst, f);
                W.mark[src] = 1;
            }
        for_entries(
            n_fork, table_ld,
            [&](uint32_t f, uint32_t c) {
                return named(f, src, dst) ? __ldcg(table + (int64_t)dst * table_ld + c) : -1;
            },
            [&](uint32_t f, uint32_t, int e) {
                if (e >= 0) W.mark[__ldg(fork_dst + f)] = 1;
            });
        __syncthreads();
        for_entries(
            n_fork, table_ld,
            [&](uint32_t f, uint32_t c) {
                return named(f, src, dst) ? __ldcg(table + (int64_t)src * table_ld + c) : -1;
            },
            [&](uint32_t f, uint32_t c, int e) {
                if (!named(f, src, dst)) return;
                if (__ldcg(W.claim + dst) != (int)f || __ldcg(W.mark + dst) != 0) {
                    set_status(status, QSA_DEV_BAD_SEQ);
                    return;
                }
                if (e >= n_pages) {
                    set_status(status, QSA_DEV_BAD_PAGE);
                    e = -1;
                }
                table[(int64_t)dst * table_ld + c] = e;
                if (e >= 0) atomicAdd(ref + e, 1);
            });
    }
    __syncthreads();

    // ---- reserve: the places to fill, in the order of (sequence, place); 1,024 sequences at a time ----
    int wanted = 0;
    for (int s0 = 0; s0 < batch; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int lo = 0, n = 0, lb = 0;
        if (s < batch) {
            lb = __ldg(len_before + s);
            const int la = __ldg(len_after + s);
            if (lb < 0 || la < lb || la > kv_capacity) {
                set_status(status, QSA_DEV_BAD_LEN);
            } else if (la > lb) {
                lo = lb / page_tokens;
                n = (la - 1) / page_tokens + 1 - lo;
            }
        }
        int total;
        s_at[tid] = block_scan(n, &total);
        s_lo[tid] = lo;
        s_lb[tid] = lb;
        __syncthreads();
        for (int c0 = 0; c0 < total; c0 += kPlanThreads) {
            const int c = c0 + tid;
            int needs = 0, e = -1;
            uint32_t place = 0;
            if (c < total) {
                int t = 0;         // the last sequence that starts at or before candidate c
#pragma unroll
                for (int step = kPlanThreads / 2; step > 0; step >>= 1)
                    if (s_at[t + step] <= c) t += step;
                const int i = s_lo[t] + (c - s_at[t]);
                place = (uint32_t)((int64_t)(s0 + t) * table_ld + i);
                e = __ldcg(table + place);
                if (e < 0 || e >= n_pages) {
                    // tokens that should be there are lost; a place that holds none yet just gets a page
                    if (e >= 0 && (int64_t)i * page_tokens < s_lb[t]) set_status(status, QSA_DEV_BAD_PAGE);
                    e = -1, needs = 1;
                } else if (__ldcg(ref + e) > 1) needs = (int64_t)i * page_tokens < s_lb[t] ? 2 : 1;
            }
            int more;
            const int rank = wanted + block_scan(needs != 0, &more);
            if (needs != 0 && rank < n_pages) {
                W.place[rank] = place | (needs == 2 ? 0x80000000u : 0u);
                W.drop[rank] = e;
            }
            wanted += more;        // at most the table's entries
        }
        __syncthreads();
    }

    // ---- the lowest free pages ----
    int found = 0;
    for (int p0 = 0; p0 < n_pages && found < wanted; p0 += kPlanThreads * 8) {
        const int base = p0 + tid * 8;
        const unsigned mask = base < n_pages ? free_mask(ref, base, n_pages) : 0u;
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

    // ---- requests are served in order while there are pages ----
    for (int r = tid; r < found; r += kPlanThreads) {
        const uint32_t place = W.place[r];
        const int to = W.free_id[r], old = W.drop[r];
        table[place & 0x7FFFFFFFu] = to;
        ref[to] = 1;               // it had no holder, so no count that was looked at changes
        if (old >= 0) atomicSub(ref + old, 1);
        if (place >> 31) W.moves[atomicAdd(&s_moves, 1)] = make_int2(old, to);
    }
    __syncthreads();
    if (tid == 0) W.head->n_moves = s_moves;
}

__global__ void __launch_bounds__(kPlanThreads)
k_pages_compact(int32_t* ref, int n_pages, PagesWork W, int32_t* n_live_out)
{
    const int tid = threadIdx.x;
    griddep_launch_dependents();
    int n_live = 0;
    unsigned first = 0;            // free pages of the first stretch, which the second pass needs again
    for (int p0 = 0; p0 < n_pages; p0 += kPlanThreads * 8) {
        const int base = p0 + tid * 8;
        const unsigned mask = base < n_pages ? free_mask(ref, base, n_pages) : 0u;
        if (p0 == 0) first = mask;
        int total;
        block_scan(base < n_pages ? min(8, n_pages - base) - __popc(mask) : 0, &total);
        n_live += total;
    }
    // k-th free id below n_live takes the k-th live id from n_live on: as many of one as of the other
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < n_pages; p0 += kPlanThreads * 8) {
        const int base = p0 + tid * 8;
        const int n = base < n_pages ? min(8, n_pages - base) : 0;
        const unsigned free = p0 == 0 ? first : n > 0 ? free_mask(ref, base, n_pages) : 0u;
        unsigned hole = 0, move = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (u >= n) continue;
            const bool is_free = free >> u & 1u;
            if (base + u < n_live) hole |= (unsigned)is_free << u;
            else if (is_free) W.remap[base + u] = -1;
            else move |= 1u << u;
        }
        // both counts of a stretch (8,192 at most) in one sum
        int total;
        const int at = block_scan(__popc(hole) | __popc(move) << 16, &total);
        int ah = holes + (at & 0xFFFF), am = movers + (at >> 16);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (hole >> u & 1u) W.moves[ah++].y = base + u;
            if (move >> u & 1u) W.moves[am++].x = base + u;
        }
        holes += total & 0xFFFF;
        movers += total >> 16;
    }
    if (tid == 0) {
        W.head->n_moves = holes;
        W.head->n_live = n_live;
        *n_live_out = n_live;
    }
    __syncthreads();
    for (int k = tid; k < holes; k += kPlanThreads) {
        const int2 mv = W.moves[k];
        W.remap[mv.x] = mv.y;
        ref[mv.y] = __ldcg(ref + mv.x);
        ref[mv.x] = 0;
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
    t.free_id = (int32_t*)take((size_t)n_pages * 4);
    t.place = (uint32_t*)take((size_t)n_pages * 4);
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
