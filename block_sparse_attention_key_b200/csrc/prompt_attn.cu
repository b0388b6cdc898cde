// Causal attention over whole prompts, packed: sequence s owns tokens
// [cu_len[s], cu_len[s+1]) of the packed arrays and token i attends the tokens of its
// own sequence up to itself,
//     out[i][h] = sum_{j <= i} softmax_j(scale q[i][h].k[j][g]) v[j][g],  g = h / G,
// G = query heads per KV head.  Below the layer's budget of 2,048 tokens the sparse
// layer is exactly this (keieiax.jp glossary "Qwen Sparse Attention", section on cost:
// dense GQA is what the sparse layer is compared with), and every prompt starts there.
//
// Work unit: one item per (query tile pair, KV head).  A query tile is 128 MMA rows, the
// floor(128 / G) consecutive tokens whose G query heads read the same K and V; an item has
// two of them (A, then B), so each K and V tile in shared memory feeds 256 rows, a
// prompt of a few tokens fills one tile with all its heads, and the causal triangle
// wastes at most one key tile per 2 x floor(128 / G) tokens.
//
// One pass over the keys with a running maximum m and sum l (exp2 domain):
//     S = Q K^T;  P = exp2(scale log2(e) S - m);  l = l f + sum P;  O = O f + P V.
// m only moves when a row's maximum grew by more than 8 (a factor of 256 in P, which
// fp32 sums and bf16 P carry without loss), so the factor f is 1 in almost every step, and
// O, which lies in TMEM, is read and written back only in the others.  An exponent is one
// multiply-add, c S - rn(c m) with c = scale log2(e): the product's rounding is one factor of the whole
// row and cancels, but from |c m| = 2^31 on it can leave fp32.  Two values of S that differ do so by
// 64 or more there after the scale, so a row above 2^30 takes the power of two below c for c, whose
// products are exact: its largest values get exponent 0 and the others at most -32.
//
// The grid has one CTA per item, but a CTA that finishes an item takes the next one off
// the queue of CTAs that have not started (cluster launch control): barriers and TMEM are
// set up once per SM, the next item's tiles load during the last steps of the current one,
// and items of very different length balance.  CTA = 12 warps, one CTA per SM (512 TMEM
// columns: S of A and B, O of A and B, 128 each; P overwrites its own S as packed bf16):
//   warp 0       takes items, finds their sequence and loads them by TMA: the two query
//                tiles, then K and V tiles of 128 tokens (32 KiB, 128-byte swizzle) through
//                a ring of 5;
//   warp 1       MMA issuer (and TMEM allocator): per key tile P_A V, S_A of the next
//                tile, P_B V, S_B of the next tile, so one tile's MMAs run while the
//                other tile's softmax does.  tcgen05 MMAs of one thread execute in
//                issue order, so S overwrites P only after P V has read it, and a
//                softmax warp that sees S knows that O holds every earlier step;
//   warps 2-3    V guard: in the key tiles that some row masks, values of V that are
//                not finite become 0 before the MMA reads them (0 x inf would put a NaN
//                into rows that must not see the token), and the first token holding
//                one is kept per dim; the epilogue gives it back to the rows behind it.
//                Each guard warp has one 64-dim half of the tile with that half's marks
//                and flag to itself, so the two never wait for each other;
//   warps 4-11   softmax, four warps per query tile, one row per thread: S from TMEM,
//                exponentials, P back to TMEM in two parts (the MMA starts on the first);
//                at the end O / l to global memory, 32 bytes per store.
// Every wait is bounded (QSA_DEV_TIMEOUT, drain, free TMEM, return).
//
// P enters P V rounded to bf16 (at most 2^-8 of it; the operands of one MMA have one type, and V is bf16), the sum
// l takes it unrounded: an output is off by 2.1e-3 of its norm at 8,192 tokens, 1.6e-3 of them its
// own rounding.
//
// Measured: 8,192 tokens at 32 / 4 heads 454 us back to back (1,211 TFLOP/s, 0.73 of a cuBLAS product's
// burst rate; tensor and special-function pipes 60% busy each).  A step of 128 keys and 256
// rows takes 3,200 cycles, 2,048 of them tensor time: a tile's S waits for its own P to be
// read, since TMEM has no room for a second S.  16 ragged prompts (5,824 tokens, 16 / 16
// heads) 48 us, 122 tokens 9.3 us.

#include <atomic>
#include <climits>

#include "sm100_host.cuh"
#include "sm100_ptx.cuh"

namespace qsa {

using namespace sm100;

namespace {

constexpr int kRows = 128;                // MMA rows of a query tile
constexpr int kKeys = 128;                // tokens of a K or V tile
constexpr int kRing = 5;                  // K and V tiles in flight
constexpr int kItems = 4;                 // items known at once: the producer's ring reaches at most three ahead
constexpr int kGuards = 4;                // masked V tiles known at once: at most three of the ring's tiles are V
constexpr int kThreads = 384;
constexpr int kReaders = 1 + 2 + 8;       // warps that read an item: MMA, guard, softmax
constexpr int kHalf = kRows * 64;         // values of one 64-dim half of a tile
constexpr uint32_t kTileBytes = kKeys * kHeadDim * 2;
constexpr uint32_t kTmemColsPrompt = 512;
constexpr uint32_t kColO = 256;           // TMEM column of O of tile A (S of A, S of B before it)
constexpr float kGrow = 8.0f;             // growth of a row maximum (log2) that rescales O
constexpr float kBig = 0x1p30f;           // scaled maximum from which a row takes a power of two for its scale
constexpr int kEarly = 3;                 // quarters of P that the MMA may read before the last one is there

enum { kPosInf = 0, kNegInf = 1, kNan = 2 };

struct Item {
    int len;                              // of the sequence; 0: no more items
    int tok0;                             // its first packed token
    int t0;                               // first token of tile A, in the sequence
    int head;                             // KV head
};

struct __align__(1024) PromptSmem {
    __nv_bfloat16 q[2][2][kHalf];         // [tile][dim half]
    __nv_bfloat16 kv[kRing][2][kHalf];    // K and V tiles in turn
    uint4 next;                           // answer of the launch control
    Item item[kItems];
    int bad[3][kHeadDim];                 // first token of the item's masked tiles whose V is +inf, -inf, NaN
    uint64_t q_full[2], q_empty[2], kv_full[kRing], kv_empty[kRing];
    uint64_t s_full[2], p_full[2][2], o_full[2];   // P in two parts
    uint64_t v_full[kGuards], v_clean[kGuards];    // masked V tiles: landed, guarded
    uint64_t item_full[kItems], item_empty[kItems], next_full, mma_done;
    uint64_t tile_done[2];                         // a tile's epilogue is over
    uint32_t tmem_base;
    int error, any_bad[2];                         // any_bad: a mark of `bad` is set, per dim half
};

// Take the next CTA of the grid that has not started; 16 bytes of answer arrive on `bar`.
__device__ __forceinline__ void take_next_cta(uint4* answer, uint64_t* bar)
{
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
            smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}

// blockIdx.x of the CTA taken, or -1 if there was none.
__device__ __forceinline__ int taken_cta(const uint4* answer)
{
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "mov.b32 %1, 0;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}\n"
        : "=r"(ok), "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return ok ? (int)x : -1;
}

__device__ __forceinline__ void store_32b(void* p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Item of grid index `cta` (index / KV heads is its place among the query tile pairs), by one
// warp; len 0 if there is none or its sequence's bounds are malformed.  Long items first:
// CTAs take them in the order of the grid, and one that starts last ends alone.
__device__ __forceinline__ Item find_item(const int32_t* __restrict__ cu, int batch, int n_tok, int n_tiles, int tq,
                                          int n_kv_heads, int cta, int lane)
{
    const int y = cta / n_kv_heads, head = cta % n_kv_heads;
    int s = -1, tile = 0;
    if (batch <= 32) {
        // every sequence in a lane: by tile number from the highest on, all sequences that have it
        int n = 0;
        if (lane < batch) {
            const int a = __ldg(cu + lane), b = __ldg(cu + lane + 1);
            if (a >= 0 && a <= b && b <= n_tok) n = (int)(((int64_t)(b - a) + tq - 1) / tq);
        }
        // tiles of number t or higher; the item's number is the largest t with more than y of them
        auto at_least = [&](int t) { return (int)__reduce_add_sync(0xffffffffu, n > t ? n - t : 0); };
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, n);
        if (y < at_least(0)) {
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                (at_least(mid) > y ? lo : hi) = mid;
            }
            tile = lo;
            const int nth = y - at_least(tile + 1);
            const unsigned has = __ballot_sync(0xffffffffu, n > tile);
            const unsigned mine = __ballot_sync(0xffffffffu, n > tile && __popc(has & ((1u << lane) - 1u)) == nth);
            s = __ffs(mine) - 1;
        }
    } else {
        // by place, from the last on.  Sequence s's tiles start at index cu[s] / tq + s, which
        // leaves every sequence at least ceil(len / tq) indices and needs no prefix sum
        const int x = n_tiles - 1 - y;
        s = find_sequence(batch, lane, [&](int i) { return __ldg(cu + i) / tq + i <= x; });
        if (s >= 0) tile = x - (__ldg(cu + s) / tq + s);
    }
    if (s < 0) return Item{0, 0, 0, head};
    const int a = __ldg(cu + s), b = __ldg(cu + s + 1);
    const int64_t first = (int64_t)tile * tq;
    if (a < 0 || a > b || b > n_tok || first < 0 || first >= b - a) return Item{0, 0, 0, head};
    return Item{b - a, a, (int)first, head};
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
k_prompt_attn(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
              const __grid_constant__ CUtensorMap tmap_v, const int32_t* __restrict__ cu_len, int batch, int n_tok,
              int n_q_heads, int n_kv_heads, int n_tiles, float scale_log2, __nv_bfloat16* __restrict__ out,
              unsigned* status)
{
    extern __shared__ uint8_t smem_raw[];
    PromptSmem& S = *reinterpret_cast<PromptSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = n_q_heads / n_kv_heads;
    const int ta = kRows / G;                              // tokens of a query tile
    const int tq = 2 * ta;

    Item it0{0, 0, 0, 0};
    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&tmap_q);
            prefetch_tensormap(&tmap_k);
            prefetch_tensormap(&tmap_v);
        }
        it0 = find_item(cu_len, batch, n_tok, n_tiles, tq, n_kv_heads, blockIdx.x, lane);
    }
    if (warp == 1) {
        tmem_alloc(&S.tmem_base, kTmemColsPrompt);
        tmem_relinquish();
    }
    if (warp == 2 && lane == 0) {
        S.error = 0;
        S.any_bad[0] = S.any_bad[1] = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.q_full[i], 1);
            mbar_init(&S.q_empty[i], 1);
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i][0], 4);                 // one arrival per softmax warp
            mbar_init(&S.p_full[i][1], 4);
            mbar_init(&S.o_full[i], 1);
            mbar_init(&S.tile_done[i], 4);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&S.kv_full[i], 1);
            mbar_init(&S.kv_empty[i], 1);
        }
        for (int i = 0; i < kGuards; ++i) {
            mbar_init(&S.v_full[i], 1);
            mbar_init(&S.v_clean[i], 2);                   // one arrival per guard warp
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&S.item_full[i], 1);
            mbar_init(&S.item_empty[i], kReaders);
        }
        mbar_init(&S.next_full, 1);
        mbar_init(&S.mma_done, 1);
        fence_mbar_init();
    }
    for (int k = tid; k < 3 * kHeadDim; k += kThreads) (&S.bad[0][0])[k] = INT_MAX;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, S.tmem_base, 0);   // the same in every lane, for the uniform datapath
    volatile int* err = &S.error;

    // What a role needs of an item.  Key tiles of A and of B (one more than A's, or as many, or
    // none); first key tile that some row masks: it and the last one are one or two tiles,
    // since an item's tokens number at most 128, or 256 from a multiple of 256 (G = 1).
    struct Tiles {
        int n_a, n_b, n_kv, j_mask;
    };
    auto tiles_of = [&](const Item& it) {
        Tiles t;
        t.n_a = (min(it.t0 + ta, it.len) - 1) / kKeys + 1;
        t.n_b = it.t0 + ta < it.len ? (min(it.t0 + 2 * ta, it.len) - 1) / kKeys + 1 : 0;
        t.n_kv = max(t.n_a, t.n_b);
        t.j_mask = it.t0 / kKeys;
        return t;
    };
    // item number n of this CTA, read by a whole warp; len 0: there are no more
    auto read_item = [&](int n, Item& it) {
        it.len = 0;
        if (!wait_phase(&S.item_full[n % kItems], (n / kItems) & 1, err, status)) return false;
        it = S.item[n % kItems];
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.item_empty[n % kItems]);
        return it.len > 0;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
        if (warp == 0) {
            // ---------------- items and loads ----------------
            Item it = it0;
            int cta = blockIdx.x, k_ring = 0, n_mask = 0, asked = 0, n_item = 0;
            bool ok = true, more = true;
            while (ok && more) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&S.next_full, 16);
                    take_next_cta(&S.next, &S.next_full);
                    // malformed lengths are skipped below and reported here: the grid has more
                    // indices than there are sequences, and each is somebody's once
                    if (cta < batch) {
                        const int a = __ldg(cu_len + cta), b = __ldg(cu_len + cta + 1);
                        if (a < 0 || a > b || b > n_tok) set_status(status, QSA_DEV_BAD_LEN);
                    }
                }
                ++asked;
                if (it.len > 0) {
                    const int slot = n_item % kItems;
                    if (n_item >= kItems && !(ok = wait_phase(&S.item_empty[slot], ((n_item / kItems) - 1) & 1, err, status)))
                        break;
                    if (lane == 0) {
                        S.item[slot] = it;
                        mbar_arrive(&S.item_full[slot]);
                    }
                    const Tiles t = tiles_of(it);
                    if (lane == 0) {
                        auto load_q = [&](int i) {
                            if (n_item > 0 && !wait_phase(&S.q_empty[i], (n_item - 1) & 1, err, status)) return false;
                            mbar_arrive_expect_tx(&S.q_full[i], (uint32_t)(ta * G) * kHeadDim * 2);
                            for (int h = 0; h < 2; ++h)
                                tma_load_3d(S.q[i][h], &tmap_q, &S.q_full[i], 64 * h, it.head * G, it.tok0 + it.t0 + i * ta);
                            return true;
                        };
                        // the first K and V ahead of the queries, whose buffers the last item still reads
                        for (int k = 0; k < 2 * t.n_kv && ok; ++k) {
                            const int ring = k_ring % kRing;
                            if (k_ring >= kRing && !(ok = wait_phase(&S.kv_empty[ring], ((k_ring / kRing) - 1) & 1, err, status)))
                                break;
                            // a masked V tile lands on a barrier of its own, which the guard can
                            // wait on without following the ring
                            const bool masked = (k & 1) && (k >> 1) >= t.j_mask;
                            uint64_t* bar = masked ? &S.v_full[n_mask % kGuards] : &S.kv_full[ring];
                            n_mask += masked;
                            mbar_arrive_expect_tx(bar, kTileBytes);
                            tma_load_4d(S.kv[ring], (k & 1) ? &tmap_v : &tmap_k, bar, 0, it.tok0 + (k >> 1) * kKeys, 0, it.head);
                            ++k_ring;
                            if (k == 1) ok = load_q(0) && load_q(1);   // also for an absent B: its barriers keep step with A's
                        }
                    }
                    ++n_item;
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                }
                if (!ok || !(ok = wait_phase(&S.next_full, (asked - 1) & 1, err, status))) break;
                cta = taken_cta(&S.next);
                fence_proxy_async();                       // read before the next answer overwrites it
                __syncwarp();
                more = cta >= 0;
                if (more) it = find_item(cu_len, batch, n_tok, n_tiles, tq, n_kv_heads, cta, lane);
            }
            if (ok) {
                const int slot = n_item % kItems;
                if (n_item < kItems || wait_phase(&S.item_empty[slot], ((n_item / kItems) - 1) & 1, err, status))
                    if (lane == 0) {
                        S.item[slot].len = 0;
                        mbar_arrive(&S.item_full[slot]);
                    }
            }
        } else if (warp == 1) {
            // ---------------- MMA ----------------
            constexpr uint32_t id_s = idesc_bf16_f32(kRows, kKeys);
            constexpr uint32_t id_o = idesc_bf16_f32(kRows, kHeadDim) | kIdescBMnMajor;
            const uint32_t me = elect_one();
            const uint64_t q_desc = smem_desc_sw128(smem_u32(S.q)), k_desc = smem_desc_sw128(smem_u32(S.kv));
            const uint64_t v_desc = smem_desc_sw128_mn(smem_u32(S.kv), kHalf * 2);
            constexpr uint32_t kTileDesc = kTileBytes >> 4, kHalfDesc = (kHalf * 2) >> 4;   // descriptor units
            auto issue_s = [&](int i, int slot) {          // S_i = Q_i K^T, 8 K steps over two 64-dim halves
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t at = (u >> 2) * kHalfDesc + 2 * (u & 3);
                    mma_bf16_ss_elected(tmem + i * kKeys, q_desc + (i * kTileDesc + at), k_desc + (slot * kTileDesc + at),
                                        id_s, u > 0, me);
                }
                mma_commit_elected(&S.s_full[i], me);
            };
            auto issue_o = [&](int i, int slot, bool first, int from, int to) {   // O_i += P_i V, K steps of 16 tokens
#pragma unroll
                for (int u = from; u < to; ++u)
                    mma_bf16_ts_elected(tmem + kColO + i * kHeadDim, tmem + i * kKeys + 8 * u,
                                        v_desc + (slot * kTileDesc + 128 * u), id_o, !first || u > 0, me);
            };
            uint32_t ring_phase = 0;                       // per slot: parity of kv_full's next use
            auto ring_full = [&](int slot) {
                const uint32_t ph = (ring_phase >> slot) & 1u;
                ring_phase ^= 1u << slot;
                return wait_phase(&S.kv_full[slot], ph, err, status);
            };
            auto after = [](int slot, int n) { return slot + n >= kRing ? slot + n - kRing : slot + n; };
            int k_slot = 0, n_mask = 0, p_phase[2] = {0, 0};
            Item it;
            bool ok = true;
            for (int n = 0; ok && read_item(n, it); ++n) {
                const Tiles t = tiles_of(it);
                ok = ring_full(k_slot);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!ok || !(ok = wait_phase(&S.q_full[i], n & 1, err, status))) continue;
                    tc_fence_after();
                    const int n_i = i ? t.n_b : t.n_a;
                    if (n_i > 0) issue_s(i, k_slot);
                    if (n_i <= 1) mma_commit_elected(&S.q_empty[i], me);
                }
                mma_commit_elected(&S.kv_empty[k_slot], me);
                for (int j = 0; j < t.n_kv && ok; ++j) {
                    const int v_slot = after(k_slot, 1), k_next = after(k_slot, 2);
                    const bool more = j + 1 < t.n_kv;
                    if (j < t.j_mask) {
                        ok = ring_full(v_slot);
                    } else {
                        const int g = n_mask++;
                        ok = wait_phase(&S.v_full[g % kGuards], (g / kGuards) & 1, err, status) &&
                             wait_phase(&S.v_clean[g % kGuards], (g / kGuards) & 1, err, status);
                    }
                    bool k_here = false;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n_i = i ? t.n_b : t.n_a;
                        if (!ok || j >= n_i) continue;
                        const uint32_t ph = (uint32_t)p_phase[i];
                        p_phase[i] ^= 1;
                        if (!(ok = wait_phase(&S.p_full[i][0], ph, err, status))) continue;
                        tc_fence_after();
                        issue_o(i, v_slot, j == 0, 0, 2 * kEarly);
                        if (more && !k_here) {
                            if (!(ok = ring_full(k_next))) continue;
                            k_here = true;
                        }
                        if (!(ok = wait_phase(&S.p_full[i][1], ph, err, status))) continue;
                        tc_fence_after();
                        issue_o(i, v_slot, j == 0, 2 * kEarly, 8);
                        if (j + 1 == n_i) {
                            mma_commit_elected(&S.o_full[i], me);
                        } else {
                            issue_s(i, k_next);
                            if (j + 2 == n_i) mma_commit_elected(&S.q_empty[i], me);
                        }
                    }
                    mma_commit_elected(&S.kv_empty[v_slot], me);
                    if (more) mma_commit_elected(&S.kv_empty[k_next], me);
                    k_slot = k_next;
                }
            }
            // every MMA issued must finish before TMEM is released
            mma_commit_elected(&S.mma_done, me);
            const uint64_t t = now_ns();
            while (!mbar_try_wait(&S.mma_done, 0) && now_ns() - t < kWaitNs) {
            }
        } else {
            // ---------------- V guard: a warp per 64-dim half (16 KiB) of each masked V tile ----------------
            const int half = warp - 2;
            int k_ring = 0, n_mask = 0, n_done_b = 0;
            bool had_b = false;
            Item it;
            for (int n = 0; read_item(n, it); ++n) {
                const Tiles t = tiles_of(it);
                // the last item's epilogues are done with `bad`.  Each tile has its own count, of the
                // items that have the tile: the warps of an absent B run ahead of A's
                bool ok = n == 0 || wait_phase(&S.tile_done[0], (n - 1) & 1, err, status);
                if (ok && had_b) ok = wait_phase(&S.tile_done[1], n_done_b++ & 1, err, status);
                if (!ok) break;
                had_b = t.n_b > 0;
                // the flag is this warp's own: every lane has read it before one clears it, and the
                // marks are cleared before the warp sets the next
                const int marked = *(volatile int*)&S.any_bad[half];
                __syncwarp();
                if (marked) {
                    for (int k = lane; k < 3 * 64; k += 32) S.bad[k >> 6][half * 64 + (k & 63)] = INT_MAX;
                    S.any_bad[half] = 0;
                    __syncwarp();
                }
                for (int j = t.j_mask; j < t.n_kv && ok; ++j) {
                    const int g = n_mask++;
                    if (!(ok = wait_phase(&S.v_full[g % kGuards], (g / kGuards) & 1, err, status))) break;
                    uint4* tile = reinterpret_cast<uint4*>(S.kv[(k_ring + 2 * j + 1) % kRing][half]);
                    bool wrote = false;
#pragma unroll 4
                    for (int c = lane; c < (int)(kTileBytes / 32); c += 32) {
                        uint4 v = tile[c];
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        uint32_t hit = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) hit |= ((w[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                        if (hit == 0) continue;
                        // chunk c: token row c >> 3, swizzled 16-byte chunk c & 7
                        const int row = c >> 3, tok = j * kKeys + row;
                        const int dim0 = half * 64 + (((c & 7) ^ (row & 7)) << 3);
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t b = (w[e >> 1] >> ((e & 1) * 16)) & 0xFFFFu;
                            if ((b & 0x7F80u) != 0x7F80u) continue;
                            const int kind = (b & 0x7Fu) ? kNan : (b & 0x8000u) ? kNegInf : kPosInf;
                            atomicMin(&S.bad[kind][dim0 + e], tok);
                            w[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
                        }
                        tile[c] = make_uint4(w[0], w[1], w[2], w[3]);
                        wrote = true;
                    }
                    if (wrote) S.any_bad[half] = 1;
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.v_clean[g % kGuards]);
                }
                if (!ok) break;
                k_ring += 2 * t.n_kv;
            }
        }
    } else {
        // ---------------- softmax ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
        const int i = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const int row_tok = row / G, row_head = row % G;   // rows past ta * G hold nothing and are not stored
        // tokens (from tile A's first) of the warp's first and last row
        const int warp_lo = i * ta + quarter * 32 / G, warp_hi = i * ta + (quarter * 32 + 31) / G;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t col_s = lanes + i * kKeys, col_o = lanes + kColO + i * kHeadDim;
        const float scale_pow2 = fmaxf(__uint_as_float(__float_as_uint(scale_log2) & 0x7F800000u), 0x1p-126f);
        const bool wide = ((uintptr_t)out & 31u) == 0;     // 32-byte stores
        int n_step = 0, n_mask = 0, n_o = 0;
        Item it;
        bool ok = true;
        for (int n = 0; ok && read_item(n, it); ++n) {
            const Tiles t = tiles_of(it);
            const int n_own = i ? t.n_b : t.n_a;
            const int first = it.t0 + i * ta;
            const int tok = first + row_tok;
            const int j_own = first / kKeys;               // first key tile this query tile masks
            n_mask += t.n_kv - t.j_mask;
            float m = -INFINITY, sc = scale_log2;          // running maximum times the row's scale, and that scale
            auto scale_for = [&](float raw) { return fabsf(raw * scale_log2) >= kBig ? scale_pow2 : scale_log2; };
            unsigned long long l2 = 0ull;                  // two partial sums
            for (int j = 0; j < n_own; ++j, ++n_step) {
                if (!(ok = wait_phase(&S.s_full[i], n_step & 1, err, status))) break;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32w(col_s + 32 * c, v[c]);
                tmem_ld_wait();
                // quarters from n_seen on are masked for the whole warp, quarters that end at or below
                // its first row's token for none of its rows; in between by element
                int n_seen = 4;
                if (j >= j_own) {
                    const int lim = tok - j * kKeys;       // keys up to lim are seen
                    const int lo = warp_lo + (it.t0 - j * kKeys), hi = warp_hi + (it.t0 - j * kKeys);
                    n_seen = min(4, hi < 0 ? 0 : hi / 32 + 1);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (32 * c + 31 > lo) {
                            const int k = lim - 32 * c;
                            const uint32_t seen = k >= 31 ? 0xFFFFFFFFu : k < 0 ? 0u : (2u << k) - 1u;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1u)) v[c][e] = 0xFF800000u;
                        }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
                    for (int e = 2; e < 32; e += 2)
                        mx[c] = max3(mx[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                }
                const float raw = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]), m_new = raw * sc;
                const bool grow = m_new > m + kGrow;
                if (j == 0) {
                    sc = scale_for(raw);
                    m = raw * sc;
                } else if (__any_sync(0xffffffffu, grow)) {
                    float f = 1.0f;
                    if (grow) {
                        // to or from a power of two the maximum grew by 32 or more: nothing is left
                        const float sc_new = scale_for(raw);
                        f = sc == scale_log2 && sc_new == scale_log2 ? exp2_approx(m - m_new) : 0.f;
                        sc = sc_new;
                        m = raw * sc;
                    }
                    l2 = fma2(l2, pack2(f, f), 0ull);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32w(col_o + 32 * c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32w(col_o + 32 * c, o);
                    }
                }
                const float neg = m == -INFINITY ? 0.f : -m;
                const unsigned long long neg2 = pack2(neg, neg), sc2 = pack2(sc, sc);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
                    if (c < n_seen) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const unsigned long long y =
                                fma2(pack2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sc2, neg2);
                            const float p0 = exp2_approx(__uint_as_float((unsigned)y));
                            const float p1 = exp2_approx(__uint_as_float((unsigned)(y >> 32)));
                            l2 = add2(l2, pack2(p0, p1));
                            p[e >> 1] = pack_bf16x2(p0, p1);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) p[e] = 0u;
                    }
                    tmem_st16w(col_s + 16 * c, p);
                    if (c == kEarly - 1 || c == 3) {
                        const int part = c == 3;
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&S.p_full[i][part]);
                    }
                }
            }
            if (!ok) break;
            if (n_own > 0) {
                const int g = n_mask - 1;                  // the item's last guarded tile: all of `bad` is there
                if (!(ok = wait_phase(&S.o_full[i], n_o & 1, err, status) &&
                           wait_phase(&S.v_clean[g % kGuards], (g / kGuards) & 1, err, status)))
                    break;
                ++n_o;
                tc_fence_after();
                const float l = __uint_as_float((unsigned)l2) + __uint_as_float((unsigned)(l2 >> 32));
                const float inv = 1.0f / l;
                const bool bad = (*(volatile int*)&S.any_bad[0] | *(volatile int*)&S.any_bad[1]) != 0;
                const bool live = row < ta * G && tok < it.len;
                char* dst = reinterpret_cast<char*>(
                    out + ((int64_t)(it.tok0 + tok) * n_q_heads + it.head * G + row_head) * kHeadDim);
                uint32_t o[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32w(col_o + 32 * c, o[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[c][e] = __float_as_uint(__uint_as_float(o[c][e]) * inv);
                if (bad) {
#pragma unroll 1
                    for (int d = 0; d < kHeadDim; ++d) {
                        const bool up = S.bad[kPosInf][d] <= tok, dn = S.bad[kNegInf][d] <= tok;
                        const float add = S.bad[kNan][d] <= tok || (up && dn) ? __uint_as_float(0x7FC00000u)
                                          : up ? INFINITY : dn ? -INFINITY : 0.f;
#pragma unroll
                        for (int u = 0; u < kHeadDim; ++u)
                            if (u == d) o[u / 32][u % 32] = __float_as_uint(__uint_as_float(o[u / 32][u % 32]) + add);
                    }
                }
                if (live) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(o[c / 2][16 * (c % 2) + 2 * e]),
                                               __uint_as_float(o[c / 2][16 * (c % 2) + 2 * e + 1]));
                        if (wide) {
                            store_32b(dst + 32 * c, w);
                        } else {
                            uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * c);
                            d4[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            d4[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.tile_done[i]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemColsPrompt);
    }
    if (tid == 0 && *err) {
        // drain after any role has given up: what is on its way into shared memory (tiles, the
        // answer about the next CTA) must land before the CTA ends (1 ms, some thousand times a
        // tile's latency)
        const uint64_t t = now_ns();
        while (now_ns() - t < 1000000) {
        }
    }
}

// ---------------------------------------------------------------- host side

int64_t prompt_attn_ctas(const qsa_dims& d, int32_t n_tok)
{
    const int tq = 2 * (kRows / (d.n_q_heads / d.n_kv_heads));
    return ((int64_t)n_tok / tq + d.batch) * d.n_kv_heads;
}

cudaError_t launch_prompt_attn(const qsa_dims& d, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                               const void* v, int64_t v_ld, const int32_t* cu_len, int32_t n_tok, void* out,
                               unsigned* status, cudaStream_t st)
{
    auto encode = encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const int G = d.n_q_heads / d.n_kv_heads;
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    CUtensorMap tq, tk, tv;
    {
        // queries [token][head][128]: a box is 64 dims of G heads of one tile's tokens
        const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)d.n_q_heads, (cuuint64_t)n_tok};
        const cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)q_ld * 2};
        const cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)(kRows / G)};
        if (encode(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    auto kv_map = [&](CUtensorMap* t, const void* p, int64_t ld) {
        // K or V as (dim of a half, token, half, head): a box is both 64-dim halves of 128 tokens
        const cuuint64_t dims[4] = {64u, (cuuint64_t)n_tok, 2u, (cuuint64_t)d.n_kv_heads};
        const cuuint64_t strides[3] = {(cuuint64_t)ld * 2, 128u, (cuuint64_t)kHeadDim * 2};
        const cuuint32_t box[4] = {64u, (cuuint32_t)kKeys, 2u, 1u};
        return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!kv_map(&tk, k, k_ld) || !kv_map(&tv, v, v_ld)) return cudaErrorInvalidValue;
    static std::atomic<bool> attr[128];
    const int smem = (int)sizeof(PromptSmem) + 1024;
    if (!set_smem_once((const void*)k_prompt_attn, smem, attr)) return cudaErrorInvalidValue;
    const int64_t ctas = prompt_attn_ctas(d, n_tok);
    const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / sqrtf((float)d.head_dim);
    k_prompt_attn<<<(unsigned)ctas, kThreads, smem, st>>>(
        tq, tk, tv, cu_len, d.batch, n_tok, d.n_q_heads, d.n_kv_heads, (int)(ctas / d.n_kv_heads),
        scale * 1.4426950408889634f, (__nv_bfloat16*)out, status);
    return cudaGetLastError();
}

}  // namespace qsa
