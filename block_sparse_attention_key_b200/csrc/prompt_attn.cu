// Causal attention over whole prompts, packed: sequence s owns tokens
// [cu_len[s], cu_len[s+1]) of the packed arrays and token i attends the tokens of its
// own sequence up to itself,
//     out[i][h] = sum_{j <= i} softmax_j(scale q[i][h].k[j][g]) v[j][g],  g = h / G,
// G = query heads per KV head.  Below the layer's budget of 2,048 tokens the sparse
// layer is exactly this (keieiax.jp glossary "Qwen Sparse Attention", section on cost:
// dense GQA is what the sparse layer is compared with), and every prompt starts there.
//
// Work unit: one CTA per (query tile pair, KV head).  A query tile is 128 MMA rows, the
// floor(128 / G) consecutive tokens whose G query heads read the same K and V; a CTA has
// two of them (A, then B), so each K and V tile in shared memory feeds 256 rows, a
// prompt of a few tokens fills one tile with all its heads, and the causal triangle
// wastes at most one key tile per 2 x floor(128 / G) tokens.
//
// One pass over the keys with a running maximum m and sum l (exp2 domain):
//     S = Q K^T;  P = exp2(scale log2(e) S - m);  l = l f + sum P;  O = O f + P V.
// m only moves when a row's maximum grew by more than 8 (a factor of 256 in P, which
// fp32 sums and bf16 P carry without loss): the factor f is 1 in almost every step, and
// O, which lies in TMEM, is read and written back only in the others.
//
// CTA = 12 warps, one CTA per SM (512 TMEM columns: S of A and B, O of A and B, 128
// each; P overwrites its own S as packed bf16):
//   warp 0       TMA producer: the two query tiles, then K and V tiles of 128 tokens
//                (32 KiB, 128-byte swizzle) through a ring of 5;
//   warp 1       MMA issuer (and TMEM allocator): per key tile P_A V, S_A of the next
//                tile, P_B V, S_B of the next tile, so one tile's MMAs run while the
//                other tile's softmax does.  tcgen05 MMAs of one thread execute in
//                issue order, so S overwrites P only after P V has read it, and a
//                softmax warp that sees S knows that O holds every earlier step;
//   warps 2-3    V guard: in the key tiles that some row masks, values of V that are
//                not finite become 0 before the MMA reads them (0 x inf would put a NaN
//                into rows that must not see the token), and the first token holding
//                one is kept per dim; the epilogue gives it back to the rows behind it;
//   warps 4-11   softmax, four warps per query tile, one row per thread: S from TMEM,
//                maximum, exponentials, P back to TMEM; at the end O / l to global
//                memory through the tile's query buffer.
// Every wait is bounded (QSA_DEV_TIMEOUT, drain, free TMEM, return).

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
constexpr int kThreads = 384;
constexpr int kHalf = kRows * 64;         // values of one 64-dim half of a tile
constexpr uint32_t kTileBytes = kKeys * kHeadDim * 2;
constexpr uint32_t kTmemColsPrompt = 512;
constexpr uint32_t kColO = 256;           // TMEM column of O of tile A (S of A, S of B before it)
constexpr float kGrow = 8.0f;             // growth of a row maximum (log2) that rescales O

enum { kPosInf = 0, kNegInf = 1, kNan = 2 };

struct __align__(1024) PromptSmem {
    __nv_bfloat16 q[2][2][kHalf];         // [tile][dim half]; the tile's output at the end
    __nv_bfloat16 kv[kRing][2][kHalf];    // K and V tiles in turn
    int bad[3][kHeadDim];                 // first token of the masked tiles whose V is +inf, -inf, NaN
    uint64_t q_full[2], kv_full[kRing], kv_empty[kRing];
    uint64_t s_full[2], p_full[2], o_full[2], mma_done;
    uint64_t v_full[2], v_clean[2];       // masked V tiles: landed, guarded
    uint32_t tmem_base;
    int error, any_bad;
    int tok0, t0, len;                    // first packed token, first token of tile A, length of the sequence
};

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
k_prompt_attn(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
              const __grid_constant__ CUtensorMap tmap_v, const int32_t* __restrict__ cu_len, int batch, int n_tok,
              int n_q_heads, int n_kv_heads, int64_t n_tiles, float scale_log2, __nv_bfloat16* __restrict__ out,
              unsigned* status)
{
    extern __shared__ uint8_t smem_raw[];
    PromptSmem& S = *reinterpret_cast<PromptSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = n_q_heads / n_kv_heads;
    const int ta = kRows / G;                              // tokens of a query tile
    const int tq = 2 * ta;
    const int head = blockIdx.x % n_kv_heads;
    const int64_t x = n_tiles - 1 - blockIdx.x / n_kv_heads;   // the longest rows of each sequence first

    if (warp == 0) {
        // sequence s's tiles start at index cu[s] / tq + s, which leaves every sequence at least
        // ceil(len / tq) indices and needs no prefix sum
        const int s = find_sequence(batch, lane, [&](int i) { return (int64_t)(__ldg(cu_len + i) / tq) + i <= x; });
        if (lane == 0) {
            int t0 = 0, len = 0, tok0 = 0;
            if (s >= 0) {
                const int a = __ldg(cu_len + s), b = __ldg(cu_len + s + 1);
                if (a >= 0 && a <= b && b <= n_tok) {
                    const int64_t first = (x - (a / tq + s)) * tq;
                    tok0 = a;
                    len = first >= 0 && first < b - a ? b - a : 0;
                    t0 = len > 0 ? (int)first : 0;
                }
            }
            S.tok0 = tok0;
            S.t0 = t0;
            S.len = len;
            S.error = 0;
            S.any_bad = 0;
            for (int i = 0; i < 2; ++i) {
                mbar_init(&S.q_full[i], 1);
                mbar_init(&S.s_full[i], 1);
                mbar_init(&S.p_full[i], 4);                // one arrival per softmax warp
                mbar_init(&S.o_full[i], 1);
                mbar_init(&S.v_full[i], 1);
                mbar_init(&S.v_clean[i], 2);               // one arrival per guard warp
            }
            for (int i = 0; i < kRing; ++i) {
                mbar_init(&S.kv_full[i], 1);
                mbar_init(&S.kv_empty[i], 1);
            }
            mbar_init(&S.mma_done, 1);
            fence_mbar_init();
        }
    }
    // malformed lengths are skipped above; the first CTA reports them
    if (blockIdx.x == 0)
        for (int s = tid; s < batch; s += kThreads) {
            const int a = __ldg(cu_len + s), b = __ldg(cu_len + s + 1);
            if (a < 0 || a > b || b > n_tok) set_status(status, QSA_DEV_BAD_LEN);
        }
    for (int k = tid; k < 3 * kHeadDim; k += kThreads) (&S.bad[0][0])[k] = INT_MAX;
    __syncthreads();
    const int len = S.len, t0 = S.t0, tok0 = S.tok0;
    if (len == 0) return;                                  // an index no tile has
    if (warp == 1) {
        tmem_alloc(&S.tmem_base, kTmemColsPrompt);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    volatile int* err = &S.error;

    // key tiles of each query tile (B may have one more than A, or none)
    const int n_a = (min(t0 + ta, len) - 1) / kKeys + 1;
    const int n_b = t0 + ta < len ? (min(t0 + 2 * ta, len) - 1) / kKeys + 1 : 0;
    const int n_kv = max(n_a, n_b);
    // first key tile that some row masks; there are one or two of them: a CTA's tokens
    // number at most 128, or 256 that start at a multiple of 256 (G = 1)
    const int j_mask = t0 / kKeys;
    // barrier that ring tile k (K_0, V_0, K_1, ...) lands on.  Masked V tiles have one each
    // that the guard can wait on without following the ring's phases; no later tile uses
    // their slots (at most three tiles come after the first of them)
    auto landed = [&](int k) {
        const int m = (k >> 1) - j_mask;
        return (k & 1) && m >= 0 ? &S.v_full[m] : &S.kv_full[k % kRing];
    };
    auto parity = [&](int k) { return (uint32_t)((k & 1) && (k >> 1) >= j_mask ? 0 : (k / kRing) & 1); };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
        if (warp == 0) {
            if (lane == 0) {
                prefetch_tensormap(&tmap_q);
                prefetch_tensormap(&tmap_k);
                prefetch_tensormap(&tmap_v);
                int issued = 0;
                auto load_q = [&](int i) {
                    mbar_arrive_expect_tx(&S.q_full[i], (uint32_t)(ta * G) * kHeadDim * 2);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(S.q[i][h], &tmap_q, &S.q_full[i], 64 * h, head * G, tok0 + t0 + i * ta);
                };
                for (int k = 0; k < 2 * n_kv; ++k) {
                    const int slot = k % kRing;
                    if (k == 0) load_q(0);
                    if (k >= kRing && !wait_phase(&S.kv_empty[slot], ((k / kRing) - 1) & 1, err, status)) break;
                    mbar_arrive_expect_tx(landed(k), kTileBytes);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(S.kv[slot][h], (k & 1) ? &tmap_v : &tmap_k, landed(k), 64 * h, head,
                                    tok0 + (k >> 1) * kKeys);
                    issued = k + 1;
                    if (k == 0 && n_b > 0) load_q(1);
                }
                if (*err) {
                    // drain: every issued tile must land before the CTA exits
                    for (int i = 0; i < (n_b > 0 ? 2 : 1); ++i) {
                        const uint64_t t = now_ns();
                        while (!mbar_try_wait(&S.q_full[i], 0) && now_ns() - t < kWaitNs) {
                        }
                    }
                    for (int k = max(0, issued - kRing); k < issued; ++k) {
                        const uint64_t t = now_ns();
                        while (!mbar_try_wait(landed(k), parity(k)) && now_ns() - t < kWaitNs) {
                        }
                    }
                }
            }
        } else if (warp == 1) {
            if (lane == 0) {
                constexpr uint32_t id_s = idesc_bf16_f32(kRows, kKeys);
                constexpr uint32_t id_o = idesc_bf16_f32(kRows, kHeadDim) | kIdescBMnMajor;
                auto issue_s = [&](int i, int k) {         // S_i = Q_i K^T, 8 K steps over two 64-dim halves
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t a = smem_desc_sw128(smem_u32(S.q[i][h]));
                        const uint64_t b = smem_desc_sw128(smem_u32(S.kv[k % kRing][h]));
#pragma unroll
                        for (int u = 0; u < 4; ++u) mma_bf16_ss(tmem + i * kKeys, a + 2 * u, b + 2 * u, id_s, h + u > 0);
                    }
                    mma_commit(&S.s_full[i]);
                };
                auto issue_o = [&](int i, int j) {         // O_i += P_i V, 8 K steps of 16 tokens
                    const uint64_t b = smem_desc_sw128_mn(smem_u32(S.kv[(2 * j + 1) % kRing][0]), kHalf * 2);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        mma_bf16_ts(tmem + kColO + i * kHeadDim, tmem + i * kKeys + 8 * u, b + 128 * u, id_o, j + u > 0);
                };
                auto ring_full = [&](int k) { return wait_phase(landed(k), parity(k), err, status); };
                bool ok = ring_full(0);
                for (int i = 0; i < (n_b > 0 ? 2 : 1) && ok; ++i)
                    if ((ok = wait_phase(&S.q_full[i], 0, err, status))) {
                        tc_fence_after();
                        issue_s(i, 0);
                    }
                mma_commit(&S.kv_empty[0]);
                for (int j = 0; j < n_kv && ok; ++j) {
                    ok = ring_full(2 * j + 1) && (j < j_mask || wait_phase(&S.v_clean[j - j_mask], 0, err, status));
                    for (int i = 0; i < 2 && ok; ++i) {
                        const int n_i = i ? n_b : n_a;
                        if (j >= n_i) continue;
                        if (!(ok = wait_phase(&S.p_full[i], j & 1, err, status))) break;
                        tc_fence_after();
                        issue_o(i, j);
                        if (j + 1 == n_i) {
                            mma_commit(&S.o_full[i]);
                        } else if ((ok = ring_full(2 * j + 2))) {
                            tc_fence_after();
                            issue_s(i, 2 * j + 2);
                        }
                    }
                    mma_commit(&S.kv_empty[(2 * j + 1) % kRing]);
                    if (j + 1 < n_kv) mma_commit(&S.kv_empty[(2 * j + 2) % kRing]);
                }
                // every MMA issued must finish before TMEM is released
                mma_commit(&S.mma_done);
                const uint64_t t = now_ns();
                while (!mbar_try_wait(&S.mma_done, 0) && now_ns() - t < kWaitNs) {
                }
            }
        } else {
            // V guard: 64 threads over the 32 KiB of each masked V tile
            const int gt = (warp - 2) * 32 + lane;
            for (int j = j_mask; j < n_kv; ++j) {
                const int k = 2 * j + 1;
                if (!wait_phase(&S.v_full[j - j_mask], 0, err, status)) break;
                uint4* tile = reinterpret_cast<uint4*>(S.kv[k % kRing][0]);
                bool wrote = false;
#pragma unroll 4
                for (int c = gt; c < (int)(kTileBytes / 16); c += 64) {
                    uint4 v = tile[c];
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t hit = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) hit |= ((w[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                    if (hit == 0) continue;
                    // chunk c: half c >> 10, token row (c >> 3) & 127, swizzled 16-byte chunk c & 7
                    const int row = (c >> 3) & 127, tok = j * kKeys + row;
                    const int dim0 = (c >> 10) * 64 + (((c & 7) ^ (row & 7)) << 3);
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
                if (wrote) S.any_bad = 1;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.v_clean[j - j_mask]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
        const int i = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const int first = t0 + i * ta;
        const int tok = first + row / G;                   // rows past ta * G hold nothing and are not stored
        const int n_own = i ? n_b : n_a;
        const int j_own = first / kKeys;                   // first key tile this query tile masks
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t col_s = lanes + i * kKeys, col_o = lanes + kColO + i * kHeadDim;
        const unsigned long long sc2 = pack2(scale_log2, scale_log2);
        float m = -INFINITY;
        unsigned long long l2 = 0ull;                      // two partial sums
        bool ok = true;
        for (int j = 0; j < n_own; ++j) {
            if (!(ok = wait_phase(&S.s_full[i], j & 1, err, status))) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32w(col_s + 32 * c, v[c]);
            tmem_ld_wait();
            if (j >= j_own) {
                const int lim = tok - j * kKeys;           // keys up to lim are seen
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * c + e > lim) v[c][e] = 0xFF800000u;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mx[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
                for (int e = 2; e < 32; e += 2) mx[c] = max3(mx[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
            }
            const float m_new = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * scale_log2;
            if (j == 0) {
                m = m_new;
            } else {
                const bool grow = m_new > m + kGrow;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? exp2_approx(m - m_new) : 1.0f;
                    if (grow) m = m_new;
                    const unsigned long long f2 = pack2(f, f);
                    l2 = fma2(l2, f2, 0ull);
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
            }
            const float neg = m == -INFINITY ? 0.f : -m;
            const unsigned long long neg2 = pack2(neg, neg);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const unsigned long long y =
                        fma2(pack2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sc2, neg2);
                    const float p0 = exp2_approx(__uint_as_float((unsigned)y));
                    const float p1 = exp2_approx(__uint_as_float((unsigned)(y >> 32)));
                    l2 = add2(l2, pack2(p0, p1));
                    p[e >> 1] = pack_bf16x2(p0, p1);
                }
                tmem_st16w(col_s + 16 * c, p);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full[i]);
        }
        if (n_own > 0 && ok && wait_phase(&S.o_full[i], 0, err, status) &&
            wait_phase(&S.v_clean[0], 0, err, status) &&
            wait_phase(&S.v_clean[n_kv - 1 - j_mask], 0, err, status)) {
            tc_fence_after();
            const float l = __uint_as_float((unsigned)l2) + __uint_as_float((unsigned)(l2 >> 32));
            const float inv = 1.0f / l;
            const bool bad = *(volatile int*)&S.any_bad != 0;
            uint8_t* stage = reinterpret_cast<uint8_t*>(S.q[i][0]);   // every S of the tile is done: its queries are free
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tmem_ld32w(col_o + 32 * c, o);
                tmem_ld_wait();
                float f[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * inv;
                if (bad) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int d = 32 * c + e;
                        const bool up = S.bad[kPosInf][d] <= tok, dn = S.bad[kNegInf][d] <= tok;
                        if (S.bad[kNan][d] <= tok || (up && dn)) f[e] = __uint_as_float(0x7FC00000u);
                        else if (up) f[e] += INFINITY;
                        else if (dn) f[e] -= INFINITY;
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    const int ch = 4 * c + (e >> 3);
                    uint4 w;
                    w.x = pack_bf16x2(f[e], f[e + 1]);
                    w.y = pack_bf16x2(f[e + 2], f[e + 3]);
                    w.z = pack_bf16x2(f[e + 4], f[e + 5]);
                    w.w = pack_bf16x2(f[e + 6], f[e + 7]);
                    *reinterpret_cast<uint4*>(stage + row * 256 + ((ch ^ (row & 15)) << 4)) = w;
                }
            }
            __syncwarp();
            // two rows per instruction, 256 contiguous bytes each
            for (int r = 0; r < 32; r += 2) {
                const int rr = quarter * 32 + r + (lane >> 4), ch = lane & 15;
                const int t = first + rr / G;
                if (rr < ta * G && t < len) {
                    const uint4 w = *reinterpret_cast<const uint4*>(stage + rr * 256 + ((ch ^ (rr & 15)) << 4));
                    uint4* dst = reinterpret_cast<uint4*>(out) +
                                 (((int64_t)tok0 + t) * n_q_heads + head * G + rr % G) * (kHeadDim / 8) + ch;
                    *dst = w;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemColsPrompt);
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
    const int ta = kRows / G;
    auto map = [&](CUtensorMap* t, const void* p, int heads, int64_t ld, int box_heads, int box_tok) {
        const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)n_tok};
        const cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)ld * 2};
        const cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tok};
        const cuuint32_t estr[3] = {1u, 1u, 1u};
        return encode(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    CUtensorMap tq, tk, tv;
    if (!map(&tq, q, d.n_q_heads, q_ld, G, ta) || !map(&tk, k, d.n_kv_heads, k_ld, 1, kKeys) ||
        !map(&tv, v, d.n_kv_heads, v_ld, 1, kKeys))
        return cudaErrorInvalidValue;
    static std::atomic<bool> attr[128];
    const int smem = (int)sizeof(PromptSmem) + 1024;
    if (!set_smem_once((const void*)k_prompt_attn, smem, attr)) return cudaErrorInvalidValue;
    const int64_t ctas = prompt_attn_ctas(d, n_tok);
    const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / sqrtf((float)d.head_dim);
    k_prompt_attn<<<(unsigned)ctas, kThreads, smem, st>>>(
        tq, tk, tv, cu_len, d.batch, n_tok, d.n_q_heads, d.n_kv_heads, ctas / d.n_kv_heads, scale * 1.4426950408889634f,
        (__nv_bfloat16*)out, status);
    return cudaGetLastError();
}

}  // namespace qsa
