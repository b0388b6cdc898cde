// Gathered GQA attention (step 4 of the QSA layer) over a cache held in 4 bits: rows of
// 128 values as 64 bytes of e2m1 codes and 8 e4m3 scales, one per 16 values,
//     k[d] = e2m1(code[d]) * e4m3(scale[d / 16])         (144 bytes of K and V per token
// and KV head instead of 512).  Same selections, draft groups, pages and results as the
// bf16 call over the cache's values.
//
// Arithmetic: a product of an e2m1 and an e4m3 number has at most 6 significant bits
// between 2^-10 and 2688, so it is exact in fp16; the hardware turns a byte of codes
// into two fp16 values and one packed multiply applies the scale.  Queries become fp16
// after a per-row power of two brings their largest magnitude to [2^14, 2^15) (a bf16
// value then keeps every bit down to 2^-31 of the row's largest, and errs by 2^-39 of it
// below); the power is undone in the logits' fp32 scale.  Probabilities are rounded to
// fp16 times 2^13 (11 bits; those below 2^-27 of the running maximum lose bits one by
// one), the sum keeps the unrounded ones.  fp32 accumulation throughout.
//
// Work unit and splits: one CTA per (split, KV head, draft group), its rows the group's
// query heads of that KV head (<= 32), tokens on the M side of mma.sync m16n8k16.  The
// splits of a (group, KV head) form one thread-block cluster and read one another's partials
// through shared memory, each finishing a share of the rows, so a call needs no scratch.
// What differs from a bf16 gather is that unpacking, not the copies, is the work (about 700
// instructions per warp and 32 tokens, 2.3 KB of each K and V), so operands never pass
// through shared memory unpacked and warps do not wait for one another: each takes 32 tokens
// at a time through a ring of its own (cp.async, four lanes per row of codes), and only the
// end is a block's.
//
// The contraction's order is free, so a lane takes 32 consecutive dims of its K rows (one
// 16-byte shared load = all A fragments of a row, the query fragments use the same order),
// and 16 consecutive dims of its V tokens (8 bytes and one scale each); V pairs are two
// tokens of one dim: their nibbles are interleaved with bit selects before the conversion
// (4 logic operations per 16 values).  The running maximum moves when it grew by more
// than 2 (probabilities then reach 2^16 / 2, inside fp16), so accumulators are rescaled,
// and lanes compare their maxima at all, in few steps.
//
// Measured: 1,024 queries of 2,052 tokens at 32 / 4 heads 263 us (issue slots 68%, ALU pipe
// 58% busy: one conversion per two values is what the format costs); a decode step of 16 x
// 64K contexts 12.2 us (18.9 MB), of one 8K context with two drafts 10.4 us: round trips and
// one pass through code that is not in the instruction cache yet.
//
// Masked places: absent tokens are zero-filled and their logits -inf.  A scale may be NaN
// (the append writes that for values that are not finite): a draft's tail token that is
// not visible to an earlier draft of its group must not reach it through 0 x NaN, so
// such groups are zeroed and the NaN is added to the rows that see the token.

#include <atomic>
#include <climits>

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace qsa {

namespace {

constexpr int kTok4 = 32;                      // tokens a warp takes at a time
constexpr int kCodeRow = kHeadDim / 2;         // 64 B of codes per token row
constexpr int kScaleRow = kHeadDim / 16;       // 8 B of scales per token row
constexpr int kCodes = kTok4 * kCodeRow;       // 2 KiB of K (or V) codes
constexpr int kScales = kTok4 * kScaleRow;
constexpr int kTile4 = 2 * (kCodes + kScales); // K codes, V codes, K scales, V scales
constexpr int kItems4 = kSelCap + 2;           // selected blocks + up to 2 tail blocks
constexpr int kItemCap4 = 576;                 // items of one split, in whole tiles
constexpr uint32_t kNoRow = 0xFFFFFFFFu;       // no such token row (a cache has fewer: the host checks)
constexpr int kMaxSplits4 = 8;                 // one cluster
constexpr float kProbShift = 13.0f;            // probabilities are held times 2^13
constexpr float kGrow4 = 2.0f;                 // growth of a row maximum (log2) that rescales the sums

struct Layout4 {
    int q, ring, tok, ioff, ipos, rowt, rows, total;
};
// `area`: bytes of the warps' rings, which the merges use at the end
__host__ __device__ inline Layout4 layout4(int rp, int warps, int depth, int area)
{
    Layout4 L;
    L.q = 0;
    L.ring = rp * kHeadDim * 2;
    L.tok = L.ring + area;
    L.ioff = L.tok + warps * depth * kTok4 * 4;
    L.ipos = L.ioff + kItemCap4 * 4;
    L.rowt = L.ipos + kItemCap4 * 4;
    L.rows = L.rowt + 32 * 4;
    L.total = L.rows + 32 * 4;
    return L;
}

__device__ __forceinline__ uint32_t swz_q(int row, int chunk)
{
    return (uint32_t)(row * (kHeadDim * 2) + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t saddr, const void* g, int src_bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(saddr), "l"(g), "r"(src_bytes));
}
__device__ __forceinline__ void cp_async8(uint32_t saddr, const void* g, int src_bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(saddr), "l"(g), "r"(src_bytes));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::); }
// (s + n) * r + kProbShift of two fp32 each
__device__ __forceinline__ float2 shifted2(unsigned long long s, unsigned long long n, unsigned long long r)
{
    const unsigned long long d = sm100::fma2(sm100::add2(s, n), r, sm100::pack2(kProbShift, kProbShift));
    return make_float2(__uint_as_float((unsigned)d), __uint_as_float((unsigned)(d >> 32)));
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the four bytes of w, each two e2m1 codes (low half first) -> four packed fp16 pairs
__device__ __forceinline__ void unpack_e2m1x8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// two e4m3 bytes (low 16 bits) -> packed fp16 pair
__device__ __forceinline__ uint32_t unpack_e4m3x2(uint32_t b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)b));
    return h;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace

// CTAs per SM that the registers have to leave room for: 128 a thread with one row tile, 168 and
// 255 with two and four.  One CTA fewer of four warps costs more than the spare registers give
// (2,368 lists of 16 rows: 259 us with two of 193, 222 us with three of 168).
constexpr int ctas_per_sm4(int nt, int warps) { return nt == 1 ? 16 / warps : warps == 4 ? (nt == 2 ? 3 : 2) : 1; }

// NT = 8-row column tiles of the MMA's N side (rows = drafts x G <= 8 * NT); KW = warps;
// D = tiles in flight per warp.
template <int NT, int KW, int D>
__global__ void __launch_bounds__(32 * KW, ctas_per_sm4(NT, KW))
k_sparse_attn_kv4(const uint4* __restrict__ q, const uint8_t* __restrict__ k_codes,
                  const uint8_t* __restrict__ k_scales, const uint8_t* __restrict__ v_codes,
                  const uint8_t* __restrict__ v_scales, const int32_t* __restrict__ q_seq,
                  const int32_t* __restrict__ q_pos, const int32_t* __restrict__ sel_idx,
                  const int32_t* __restrict__ sel_cnt, const int32_t* __restrict__ page_table, int page_tokens,
                  int64_t table_ld, int64_t n_pages, int batch, int n_q_heads, int n_kv_heads, int64_t kv_capacity,
                  int bs_log2, int top_k, int group_q, float scale_log2, int items_per_split, int n_split, int area,
                  __nv_bfloat16* __restrict__ out, unsigned* status)
{
    constexpr int RP = 8 * NT;           // padded rows
    constexpr int kT = 32 * KW;          // threads
    constexpr int kPerT = (kItemCap4 + kT - 1) / kT;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int s_cnt, s_nitems, s_seq, s_nc0, s_tlast;
    const Layout4 SL = layout4(RP, KW, D, area);
    const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
    uint32_t* s_ioff = reinterpret_cast<uint32_t*>(smem + SL.ioff);
    int* s_ipos = reinterpret_cast<int*>(smem + SL.ipos);
    int* s_rowt = reinterpret_cast<int*>(smem + SL.rowt);
    float* s_rows = reinterpret_cast<float*>(smem + SL.rows);

    // grid (splits, KV heads, groups), or (groups, KV heads) for one CTA per pair
    const bool one = n_split == 1;
    const int split = one ? 0 : blockIdx.x, g = blockIdx.y, grp = one ? blockIdx.x : blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = n_q_heads / n_kv_heads;
    const int R = group_q * G;
    const int64_t qi0 = (int64_t)grp * group_q;
    const int bs = 1 << bs_log2;     // tokens per block
    const int ipt = kTok4 >> bs_log2;  // blocks per tile

    // ---- one round of independent loads: positions, queries, this split's selection ----
    const int a0 = split * items_per_split;
    int raw[kPerT];
#pragma unroll
    for (int u = 0; u < kPerT; ++u) {
        const int k = tid + u * kT;
        const int a = a0 + k;
        raw[u] = (k < items_per_split && a < kSelCap) ? __ldg(sel_idx + (int64_t)grp * kSelCap + a) : -1;
    }
    const int cnt_raw = tid == 0 ? __ldg(sel_cnt + grp) : 0;
    if (warp == 0) {
        // lane r < RP: row r = (draft query j = r / G, head r % G); its position, or -2
        const int64_t qi = qi0 + (lane < R ? lane / G : 0);
        const int s0 = __ldg(q_seq + qi0), t0 = __ldg(q_pos + qi0), sj = __ldg(q_seq + qi), tj = __ldg(q_pos + qi);
        const bool ok0 = s0 >= 0 && s0 < batch && t0 >= 0 && (int64_t)t0 < kv_capacity;
        const int nc0 = ok0 ? (int)(((int64_t)t0 + 1) >> bs_log2) : 0;
        int t = -2;
        if (lane < R && ok0) {
            // a draft query follows the selection's query within the two tail blocks
            const bool ok = sj == s0 && tj >= t0 && (int64_t)tj <= (int64_t)bs * nc0 + 2 * bs - 1 &&
                            (int64_t)tj < kv_capacity;
            if (ok) t = tj;
            else if (split == 0 && g == 0 && lane % G == 0)
                set_status(status, sj != s0 ? QSA_DEV_BAD_SEQ : QSA_DEV_BAD_POS);
        }
        if (lane < RP) s_rowt[lane] = t;
        const int tl = __reduce_max_sync(0xffffffffu, lane < R ? t : -2);
        if (lane == 0) {
            s_seq = ok0 ? s0 : -1;
            s_nc0 = nc0;
            s_tlast = tl;
            if (!ok0 && split == 0 && g == 0)
                set_status(status, (s0 < 0 || s0 >= batch) ? QSA_DEV_BAD_SEQ : QSA_DEV_BAD_POS);
        }
    }
    // query rows in fp16, 16 threads per row: the row's largest magnitude goes to [2^14, 2^15);
    // by the last warps, beside the first one's loads
    for (int k = kT - 1 - tid; k < RP * 16; k += kT) {
        const int row = k >> 4, ch = k & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < R) v = __ldg(q + ((qi0 + row / G) * n_q_heads + (int64_t)g * G + row % G) * 16 + ch);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0;            // largest exponent field (bits 14..7 of a bf16)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7F80u, (w[e] >> 16) & 0x7F80u));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // exponent e (value 2^(e - 127) to 2^(e - 126)): times 2^(141 - e), kept a normal fp32 number
        const int up = min(max(141 - (int)(top >> 7), -113), 100);
        const float f = __int_as_float((127 + up) << 23);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = pack_f16(bf16lo(w[e]) * f, bf16hi(w[e]) * f);
        *reinterpret_cast<uint4*>(smem + swz_q(row, ch)) = make_uint4(h[0], h[1], h[2], h[3]);
        // (not 0: a masked logit of -inf stays it; what is below 2^-126 makes every exponent 0 anyway)
        if (ch == 0) s_rows[row] = fmaxf(__int_as_float((127 - up) << 23) * scale_log2, 0x1p-126f);
    }
    __syncthreads();  // s_seq, s_nc0, s_tlast, s_rowt, query rows
    if (tid == 0) {
        int cnt = s_seq >= 0 ? cnt_raw : 0;
        const int cnt_max = min(s_nc0, top_k);
        if (cnt < 0 || cnt > cnt_max) {
            if (split == 0 && g == 0) set_status(status, QSA_DEV_BAD_SEL);
            cnt = cnt < 0 ? 0 : cnt_max;
        }
        const int tl = s_tlast;
        const int64_t tail0 = (int64_t)bs * s_nc0;
        const int n_tail = tl >= tail0 ? (int)((tl - tail0) >> bs_log2) + 1 : 0;
        s_cnt = cnt;
        s_nitems = cnt + n_tail;
    }
    __syncthreads();
    const int cnt = s_cnt;
    const int n_blk = max(0, min(a0 + items_per_split, s_nitems) - a0);
    const int s = s_seq;
    const int nc0 = s_nc0;
#pragma unroll
    for (int u = 0; u < kPerT; ++u) {
        const int k = tid + u * kT;
        if (k >= n_blk) continue;
        const int a = a0 + k;
        int p0 = -1, ipos = -1;  // first token of the item; ipos -1: visible to every row
        if (a < cnt) {
            const int b = raw[u];
            if (b >= 0 && b < nc0) p0 = b << bs_log2;
            else set_status(status, QSA_DEV_BAD_SEL);
        } else {
            p0 = (nc0 + (a - cnt)) << bs_log2;
            ipos = p0;
        }
        uint32_t off = kNoRow;   // token row in the cache
        if (p0 >= 0) {
            if (page_table) {
                const int page = __ldg(page_table + (int64_t)s * table_ld + p0 / page_tokens);
                if (page >= 0 && page < n_pages)
                    off = ((uint32_t)page * n_kv_heads + g) * page_tokens + p0 % page_tokens;
                else
                    set_status(status, QSA_DEV_BAD_PAGE);
            } else {
                off = ((uint32_t)s * n_kv_heads + g) * (uint32_t)kv_capacity + p0;
            }
        }
        s_ioff[k] = off;
        s_ipos[k] = ipos;
    }
    __syncthreads();

    const int tlast = s_tlast;
    const int n_tiles = (n_blk + ipt - 1) / ipt;
    const uint32_t ring = sbase + SL.ring + warp * (D * kTile4);
    const uint8_t *k_lane = k_codes + (lane & 3) * 16, *v_lane = v_codes + (lane & 3) * 16;
    int* s_tok = reinterpret_cast<int*>(smem + SL.tok) + warp * (D * kTok4);
    // One tile into a slot of the warp's ring; returns whether some token of it is absent or
    // not visible to every row (then the tokens' positions are in s_tok).
    auto load_tile = [&](int tile, int slot) {
        const uint32_t st = ring + slot * kTile4;
        // lane = token row: its place in the cache, its scales
        const int it = tile * ipt + (lane >> bs_log2), tin = lane & (bs - 1);
        uint32_t e = kNoRow;
        int tp = INT_MAX;
        if (it < n_blk) {
            e = s_ioff[it];
            const int ip = s_ipos[it];
            if (ip >= 0 && ip + tin > tlast) e = kNoRow;   // past the group's last draft token
            if (e != kNoRow) {
                e += tin;
                tp = ip < 0 ? -1 : ip + tin;
            }
        }
        // four lanes per row, a 16-byte chunk of K and of V codes each; the upper bit of V's
        // chunk is flipped every two tokens, so that the reads below meet no bank twice
        const uint32_t kd = st + (lane >> 2) * 64 + (lane & 3) * 16;
        const uint32_t vd = st + kCodes + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 2) & 2)) << 4);
        auto copy = [&](uint32_t row, int u, int n16) {
            const uint64_t at = (uint64_t)row * kCodeRow;
            cp_async16(kd + 512 * u, k_lane + at, n16);
            cp_async16(vd + 512 * u, v_lane + at, n16);
        };
        if (__all_sync(0xffffffffu, e != kNoRow)) {
            cp_async8(st + 2 * kCodes + lane * 8, k_scales + (uint64_t)e * kScaleRow, 8);
            cp_async8(st + 2 * kCodes + kScales + lane * 8, v_scales + (uint64_t)e * kScaleRow, 8);
#pragma unroll
            for (int u = 0; u < 4; ++u) copy(__shfl_sync(0xffffffffu, e, (lane >> 2) + 8 * u), u, 16);
        } else {
            // absent tokens are filled with zeros
            const uint64_t es = e != kNoRow ? e : 0u;
            cp_async8(st + 2 * kCodes + lane * 8, k_scales + es * kScaleRow, e != kNoRow ? 8 : 0);
            cp_async8(st + 2 * kCodes + kScales + lane * 8, v_scales + es * kScaleRow, e != kNoRow ? 8 : 0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t er = __shfl_sync(0xffffffffu, e, (lane >> 2) + 8 * u);
                copy(er != kNoRow ? er : 0u, u, er != kNoRow ? 16 : 0);
            }
        }
        cp_commit();
        const bool special = __any_sync(0xffffffffu, tp != -1);
        if (special) s_tok[slot * kTok4 + lane] = tp;
        return special;
    };

    unsigned special = 0;            // bit per slot
#pragma unroll
    for (int u = 0; u < D; ++u) {
        const int t = warp + u * KW;
        if (t < n_tiles) special |= (unsigned)load_tile(t, u) << u;
        else cp_commit();
    }

    const int c4 = lane & 3, l4 = lane >> 2;
    int trow[NT][2];
    float rsc[NT][2];                // logit scale of the lane's accumulator columns
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            trow[nt][j] = s_rowt[8 * nt + 2 * c4 + j];
            rsc[nt][j] = s_rows[8 * nt + 2 * c4 + j];
        }
    // Q^T fragments (B operand: k = dims, n = rows): the lane holds dims 32 c4 .. 32 c4 + 31 of
    // row 8 nt + l4, 4 dims per k-step; in registers for NT <= 2
    constexpr bool kHoldQ = NT <= 2;
    uint32_t qb[kHoldQ ? 4 : 1][NT][4];
    if constexpr (kHoldQ) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint4 v = lds128(sbase + swz_q(8 * nt + l4, 4 * c4 + w));
                qb[w][nt][0] = v.x, qb[w][nt][1] = v.y, qb[w][nt][2] = v.z, qb[w][nt][3] = v.w;
            }
    }

    float o[8][NT][4];
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
    // running maxima before the logit scale, so that an exponent is the scaled difference of two
    // products: exactly 0 at the maximum however large the logits are.  neg: -m, of the maximum 0
    // while there is none
    float m[NT][2], l[NT][2], neg[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f, neg[nt][0] = neg[nt][1] = 0.f;
    // token (of 16) of MMA row r, in either half of a tile: r / 2 for even r, 4 + (r / 2 ^ 1) for
    // odd r, + 8 for rows 8 and up.  Two neighbouring rows lie in different halves of 128 bytes
    // (K's reads), the even rows are tokens 0 to 3 (V's reads)
    const int tk = l4 & 1 ? 4 + ((l4 >> 1) ^ 1) : l4 >> 1;
    const int tv0 = c4, tv1 = 4 + (c4 ^ 1);   // of rows 2 c4 and 2 c4 + 1
    const uint32_t k_at = tk * 64 + c4 * 16, ks_at = 2 * kCodes + tk * 8 + 2 * c4;
    const uint32_t v_at = kCodes + (((l4 >> 1) ^ (c4 & 2)) << 4) + (l4 & 1) * 8, vs_at = 2 * kCodes + kScales + l4;
    const uint32_t v_at0 = v_at + tv0 * 64, v_at1 = v_at + tv1 * 64;   // (tv0 and tv1 have the same bit 1)
    const uint32_t vs_at0 = vs_at + tv0 * 8, vs_at1 = vs_at + tv1 * 8;

    int slot = 0;
    for (int t = warp; t < n_tiles; t += KW) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(D - 1));
        __syncwarp();
        const uint32_t st = ring + slot * kTile4;
        const bool masked = special >> slot & 1u;
        // ---- S^T = K Q^T: rows l4 and l4 + 8 of each half, dims 32 c4 + 8 w .. + 7 per word ----
        float sc[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[h][nt][e] = 0.f;
            const uint4 k0 = lds128(st + k_at + 1024 * h), k1 = lds128(st + k_at + 1024 * h + 512);
            const uint32_t s0 = unpack_e4m3x2(lds16(st + ks_at + 128 * h)), s1 = unpack_e4m3x2(lds16(st + ks_at + 128 * h + 64));
            const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                // words 0 and 1 lie in the lane's first scale group, 2 and 3 in its second
                const uint32_t f0 = __byte_perm(s0, s0, w < 2 ? 0x1010 : 0x3232);
                const uint32_t f1 = __byte_perm(s1, s1, w < 2 ? 0x1010 : 0x3232);
                uint32_t h0[4], h1[4];
                unpack_e2m1x8(kw0[w], h0);
                unpack_e2m1x8(kw1[w], h1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h0[e] = mul_f16x2(h0[e], f0);
                    h1[e] = mul_f16x2(h1[e], f1);
                }
                const uint32_t ka[4] = {h0[0], h1[0], h0[1], h1[1]};
                const uint32_t kb[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (kHoldQ) {
                        mma16816_f16(sc[h][nt], ka, qb[w][nt][0], qb[w][nt][1]);
                        mma16816_f16(sc[h][nt], kb, qb[w][nt][2], qb[w][nt][3]);
                    } else {
                        const uint4 v = lds128(sbase + swz_q(8 * nt + l4, 4 * c4 + w));
                        mma16816_f16(sc[h][nt], ka, v.x, v.y);
                        mma16816_f16(sc[h][nt], kb, v.z, v.w);
                    }
                }
            }
        }
        // ---- softmax: element e of half h: token 16 h + tk (+8 for e >= 2), row 8nt + 2c4 + (e & 1) ----
        if (masked) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int tp0 = s_tok[slot * kTok4 + 16 * h + tk], tp1 = s_tok[slot * kTok4 + 16 * h + tk + 8];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((e < 2 ? tp0 : tp1) > trow[nt][e & 1]) sc[h][nt][e] = -INFINITY;
            }
        }
        float mx[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // of the lane's tokens; of all 32 only where some lane's maximum grew
                mx[nt][j] = fmaxf(fmaxf(sc[0][nt][j], sc[0][nt][j + 2]), fmaxf(sc[1][nt][j], sc[1][nt][j + 2]));
                grow = grow || (mx[nt][j] - m[nt][j]) * rsc[nt][j] > kGrow4;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = mx[nt][j];
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const bool g_ = (x - m[nt][j]) * rsc[nt][j] > kGrow4;
                    const float f = g_ ? exp2_approx((m[nt][j] - x) * rsc[nt][j]) : 1.0f;
                    if (g_) {
                        m[nt][j] = x;
                        neg[nt][j] = -x;
                    }
                    l[nt][j] *= f;
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt) {
                        o[mt][nt][j] *= f;
                        o[mt][nt][j + 2] *= f;
                    }
                }
        }
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const unsigned long long r2 = sm100::pack2(rsc[nt][0], rsc[nt][1]), n2 = sm100::pack2(neg[nt][0], neg[nt][1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 a = shifted2(sm100::pack2(sc[h][nt][0], sc[h][nt][1]), n2, r2);
                const float2 b = shifted2(sm100::pack2(sc[h][nt][2], sc[h][nt][3]), n2, r2);
                const float p0 = exp2_approx(a.x), p1 = exp2_approx(a.y);
                const float p2 = exp2_approx(b.x), p3 = exp2_approx(b.y);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pb[h][nt][0] = movm_t(pack_f16(p0, p1));  // MMA rows 0-7 -> B operand (k = token, n = row)
                pb[h][nt][1] = movm_t(pack_f16(p2, p3));  // rows 8-15
            }
        }
        // ---- O^T += V^T P^T: token pairs (tv0, tv1) and (tv0 + 8, tv1 + 8) of each half ----
        int bad = INT_MAX;           // first tail token whose group l4 is NaN
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint2 vw[4];
            uint32_t vs[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int rows = 16 * h + (u & 2 ? 8 : 0);
                vw[u] = lds64(st + (u & 1 ? v_at1 : v_at0) + rows * 64);
                vs[u] = lds8(st + (u & 1 ? vs_at1 : vs_at0) + rows * 8);
                if (masked && group_q > 1) {
                    const int tp = s_tok[slot * kTok4 + rows + (u & 1 ? tv1 : tv0)];
                    if (tp >= 0 && tp != INT_MAX && (vs[u] & 0x7Fu) == 0x7Fu) {
                        bad = min(bad, tp);
                        vs[u] = 0;
                    }
                }
            }
            const uint32_t g0 = unpack_e4m3x2(vs[0] | (vs[1] << 8)), g1 = unpack_e4m3x2(vs[2] | (vs[3] << 8));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // 8 dims 16 l4 + 8 half + i: nibble pairs (token A, token B) of dim i in byte order
                const uint32_t a = half ? vw[0].y : vw[0].x, b = half ? vw[1].y : vw[1].x;
                const uint32_t c = half ? vw[2].y : vw[2].x, d = half ? vw[3].y : vw[3].x;
                constexpr uint32_t kLow = 0x0F0F0F0Fu;
                uint32_t e0[4], e1[4], d0[4], d1[4];   // even dims, odd dims of the two token pairs
                unpack_e2m1x8((a & kLow) | ((b << 4) & ~kLow), e0);
                unpack_e2m1x8(((a >> 4) & kLow) | (b & ~kLow), d0);
                unpack_e2m1x8((c & kLow) | ((d << 4) & ~kLow), e1);
                unpack_e2m1x8(((c >> 4) & kLow) | (d & ~kLow), d1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // MMA row l4: dim 16 l4 + 2 mt, row l4 + 8: dim 16 l4 + 2 mt + 1
                    const int mt = 4 * half + i;
                    const uint32_t va[4] = {mul_f16x2(e0[i], g0), mul_f16x2(d0[i], g0), mul_f16x2(e1[i], g1),
                                            mul_f16x2(d1[i], g1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[mt][nt], va, pb[h][nt][0], pb[h][nt][1]);
                }
            }
        }
        if (masked && group_q > 1) {
            bad = min(bad, __shfl_xor_sync(0xffffffffu, bad, 1));
            bad = min(bad, __shfl_xor_sync(0xffffffffu, bad, 2));
            if (bad != INT_MAX) {
#pragma unroll
                for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (trow[nt][e & 1] >= bad) o[mt][nt][e] = __int_as_float(0x7FC00000);
            }
        }
        __syncwarp();                // every lane is done with the slot
        special &= ~(1u << slot);
        if (t + D * KW < n_tiles) special |= (unsigned)load_tile(t + D * KW, slot) << slot;
        else cp_commit();
        slot = slot + 1 == D ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;\n" ::);
    __syncthreads();

    // ---- merge the warps: (m, l) per row, O^T into shared memory (ring area) ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
            l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
        }
    // O in 16-byte pieces, piece c of row r at place c ^ (r / 2 & 3): eight lanes that store together
    // hold rows 2 c4 + j and pieces 4 l4 + n of two l4, which are then in different banks
    float4* s_o = reinterpret_cast<float4*>(smem + SL.ring);  // [KW][RP][32]
    float* s_m = reinterpret_cast<float*>(s_o + KW * RP * 32);  // [KW][RP]
    float* s_l = s_m + KW * RP;                                 // [KW][RP]
    auto piece = [](int row, int c) { return row * 32 + (c ^ (row >> 1 & 3)); };
    if (l4 == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s_m[warp * RP + 8 * nt + 2 * c4 + j] = m[nt][j];
                s_l[warp * RP + 8 * nt + 2 * c4 + j] = l[nt][j];
            }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // 16 consecutive dims of one row per lane
            const int row = 8 * nt + 2 * c4 + j;
#pragma unroll
            for (int mt = 0; mt < 8; mt += 2)
                s_o[warp * RP * 32 + piece(row, 4 * l4 + mt / 2)] =
                    make_float4(o[mt][nt][j], o[mt][nt][j + 2], o[mt + 1][nt][j], o[mt + 1][nt][j + 2]);
        }
    __syncthreads();

    // ---- merge the warps: a thread per row and 4 dims ----
    namespace cg = cooperative_groups;
    constexpr int kPieces = RP * 32;
    float4* s_mo = s_o;                                       // [RP][32] merged, in the place of warp 0's
    float* s_mm = reinterpret_cast<float*>(smem + SL.tok);    // [RP], [RP] merged (the positions are no longer needed)
    float* s_ml = s_mm + RP;
    for (int k = tid; k < kPieces; k += kT) {
        const int row = k >> 5, c = k & 31;
        const float r = s_rows[row];
        float M = -INFINITY;
#pragma unroll 4
        for (int w = 0; w < KW; ++w) M = fmaxf(M, s_m[w * RP + row]);
        const float Mu = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < KW; ++w) {
            const float f = exp2_approx((s_m[w * RP + row] - Mu) * r);
            const float4 v = s_o[w * kPieces + piece(row, c)];
            L += s_l[w * RP + row] * f;
            acc.x += v.x * f;
            acc.y += v.y * f;
            acc.z += v.z * f;
            acc.w += v.w * f;
        }
        s_mo[piece(row, c)] = acc;       // read by this thread alone so far
        if (c == 0) {
            s_mm[row] = M;
            s_ml[row] = L;
        }
    }

    // ---- merge the splits: each CTA of the cluster finishes its share of the pieces ----
    auto store = [&](int row, int c, float4 a, float L) {
        if (row >= R) return;
        const float inv = L == 0.f ? 0.f : 1.f / L;   // a row that attends nothing is 0; a NaN sum stays NaN
        uint2 v = make_uint2(0u, 0u);                 // and so is one of a skipped query
        if (s_rowt[row] >= 0) {
            v.x = pack_bf16x2(a.x * inv, a.y * inv);
            v.y = pack_bf16x2(a.z * inv, a.w * inv);
        }
        *reinterpret_cast<uint2*>(out + ((qi0 + row / G) * n_q_heads + (int64_t)g * G + row % G) * kHeadDim + 4 * c) = v;
    };
    if (n_split == 1) {
        __syncthreads();
        for (int k = tid; k < kPieces; k += kT) store(k >> 5, k & 31, s_mo[piece(k >> 5, k & 31)], s_ml[k >> 5]);
        return;
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    // `width` lanes per piece, one per split, so that a share takes one round trip to the others
    const int width = n_split <= 2 ? 2 : n_split <= 4 ? 4 : 8;
    const int sp = tid & (width - 1);
    for (int k0 = 0; k0 < kPieces; k0 += kT / width * n_split) {
        const int k = k0 + tid / width * n_split + split;
        const int row = k >> 5, c = k & 31;
        float M = -INFINITY, L = 0.f, r = 1.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (sp < n_split && k < kPieces) {
            r = s_rows[row];     // the same in every split
            M = *cl.map_shared_rank(s_mm + row, sp);
            L = *cl.map_shared_rank(s_ml + row, sp);
            acc = *cl.map_shared_rank(s_mo + piece(row, c), sp);
        }
        float Mg = M;
        for (int o = width >> 1; o > 0; o >>= 1) Mg = fmaxf(Mg, __shfl_xor_sync(0xffffffffu, Mg, o));
        const float f = exp2_approx((M - (Mg == -INFINITY ? 0.f : Mg)) * r);
        L *= f;
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
        for (int o = width >> 1; o > 0; o >>= 1) {
            L += __shfl_xor_sync(0xffffffffu, L, o);
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
        }
        if (sp == 0 && k < kPieces) store(row, c, acc, L);
    }
    cl.sync();   // nobody's shared memory goes before all have read it
}

// ---------------------------------------------------------------- host side

namespace {

int nt_for(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

// One kernel per row tile count and call size (lists = query groups x KV heads).  Few lists:
// one CTA per SM (or a cluster per list), as many warps as its registers allow.  More: smaller
// CTAs, several per SM, whose starts and ends overlap and whose last wave is shorter.  Lists of
// 2,052 tokens, us:
//   <= 8 rows, 8 / 4 / 2 warps: 148 lists 16.8 / 21.4 / 39.5, 296 lists 24.7 / 27.5 / 40.4,
//   400 lists 36.4 / 35.1 / 49.5, 4,096 lists 283 / 261 / 255; 16 warps (measured with a loop
//   about 3% slower): 15.6, 29.4, 42.1 and 371
//   <= 16 rows, 8 / 4 / 2 warps: 148 lists 20.6 / 28.6 / 43.2, 149 lists 37.3 / 35.4 / 43.5,
//   400 lists 56.6 / 45.1 / 58.0, 2,368 lists 294 / 222 / 224
//   <= 32 rows, 8 / 4 / 2 warps: 148 lists 33.3 / 41.9 / 72.5, 149 lists 59.9 / 52.7 / 73.3,
//   400 lists 92 / 90 / 97, 2,368 lists 483 / 405 / 384
// Two warps were only tried: the 2 to 5% that they are ahead at thousands of lists are paid for by
// up to 40% at 150 to 400, and a third kernel per row tile count would have to be kept for them.
int tier4(int64_t lists) { return lists <= 148 ? 0 : lists <= 296 ? 1 : 2; }

struct Shape {
    const void* fn;
    int warps, depth;
};
Shape shape4(int nt, int tier)
{
    if (nt == 1)
        return tier == 0   ? Shape{(const void*)k_sparse_attn_kv4<1, 16, 2>, 16, 2}
               : tier == 1 ? Shape{(const void*)k_sparse_attn_kv4<1, 8, 2>, 8, 2}
                           : Shape{(const void*)k_sparse_attn_kv4<1, 4, 2>, 4, 2};
    if (nt == 2)
        return tier == 0 ? Shape{(const void*)k_sparse_attn_kv4<2, 8, 2>, 8, 2}
                         : Shape{(const void*)k_sparse_attn_kv4<2, 4, 2>, 4, 2};
    return tier == 0 ? Shape{(const void*)k_sparse_attn_kv4<4, 8, 2>, 8, 2}
                     : Shape{(const void*)k_sparse_attn_kv4<4, 4, 2>, 4, 2};
}

constexpr int kMaxArea = 160 * 1024;   // of the rings and merge buffers

int shape_index(int nt, int tier) { return (nt == 1 ? 0 : nt == 2 ? 1 : 2) + 3 * tier; }

bool configure4(int dev, int nt, int tier)
{
    static std::atomic<bool> done[64][9];
    if (dev < 0 || dev >= 64) return false;
    std::atomic<bool>& d = done[dev][shape_index(nt, tier)];
    if (d.load()) return true;
    const Shape s = shape4(nt, tier);
    if (cudaFuncSetAttribute(s.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             layout4(8 * nt, s.warps, s.depth, kMaxArea).total) != cudaSuccess)
        return false;
    d.store(true);
    return true;
}

int area4(int rp, const Shape& s)
{
    // the rings, then the warps' partials
    const int parts = s.warps * rp * (kHeadDim + 2) * 4, rings = s.warps * s.depth * kTile4;
    return rings > parts ? rings : parts;
}

}  // namespace

// Splits of `pairs` lists: as many as still run all at once.  Clusters stay inside a group of
// SMs (16 to 18 of them on a B200), so fewer fit than the SM count says: 8 splits of 16 pairs
// took 15.0 us where 6 took 8.5 (8 query heads, one list of 2,048 tokens per pair); from 8
// splits on (8.1 us for one pair) more of them gain nothing.  The device's answer per split
// count is kept; without a device every SM counts.
static int splits_at_once(int dev, int nt, int64_t pairs, const Shape& s, int smem)
{
    static std::atomic<int> fits[64][3][kMaxSplits4 + 1];   // clusters + 1; 0: not asked yet
    for (int ns = kMaxSplits4; ns > 1; --ns) {
        if (pairs * ns > 148) continue;
        if (dev < 0 || dev >= 64) return ns;
        std::atomic<int>& f = fits[dev][shape_index(nt, false)][ns];
        int n = f.load();
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)ns, 1, 1);
            cfg.blockDim = dim3((unsigned)(32 * s.warps));
            cfg.dynamicSmemBytes = (size_t)smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)ns;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int clusters = 0;
            if (cudaOccupancyMaxActiveClusters(&clusters, s.fn, &cfg) != cudaSuccess) {
                cudaGetLastError();
                clusters = 0;
            }
            n = clusters + 1;
            f.store(n);
        }
        if (n - 1 >= pairs) return ns;
    }
    return 1;
}

void plan_kv4(const qsa_dims& d, int64_t n_groups, int group_q, qsa_attn_plan_info* p)
{
    const int rows = d.n_q_heads / d.n_kv_heads * group_q;
    const int nt = nt_for(rows), rp = 8 * nt;
    const int64_t pairs = n_groups * d.n_kv_heads;
    const int tier = tier4(pairs);
    const Shape s = shape4(nt, tier);
    const int smem = layout4(rp, s.warps, s.depth, area4(rp, s)).total;
    const int ipt = kTok4 / d.block_size;
    const int tiles_max = (kItems4 + ipt - 1) / ipt;   // 17 to 257
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || !configure4(dev, nt, tier)) {
        cudaGetLastError();
        dev = -1;
    }
    int ns = tier > 0 ? 1 : splits_at_once(dev, nt, pairs, s, smem);
    const int tiles = (tiles_max + ns - 1) / ns;
    ns = (tiles_max + tiles - 1) / tiles;          // no split without a tile
    p->n_split = ns;
    p->n_stages = s.warps * s.depth;
    p->threads = 32 * s.warps;
    p->smem_bytes = smem;
    p->ctas = pairs * ns;
    p->cluster_merge = ns > 1;
    p->rows = rows;
}

cudaError_t launch_sparse_attn_kv4(const qsa_dims& d, const qsa_kv4_cache& c, const void* q, const int32_t* q_seq,
                                   const int32_t* q_pos, const int32_t* sel_idx, const int32_t* sel_cnt,
                                   int64_t n_groups, int group_q, void* out, unsigned* status, cudaStream_t st)
{
    if (n_groups <= 0) return cudaSuccess;
    qsa_attn_plan_info p;
    plan_kv4(d, n_groups, group_q, &p);
    const int nt = nt_for(p.rows);
    const int tier = tier4(n_groups * d.n_kv_heads);
    int bs_log2 = 0;
    while ((1 << bs_log2) < d.block_size) ++bs_log2;
    const int n_split = p.n_split, ipt = kTok4 >> bs_log2;
    const int tiles_max = (kItems4 + ipt - 1) / ipt;
    const int items = (tiles_max + n_split - 1) / n_split * ipt;   // of one split, in whole tiles
    const int area = area4(8 * nt, shape4(nt, tier));
    const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / sqrtf((float)d.head_dim);

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = n_split == 1 ? dim3((unsigned)n_groups, (unsigned)d.n_kv_heads, 1u)
                               : dim3((unsigned)n_split, (unsigned)d.n_kv_heads, (unsigned)n_groups);
    cfg.blockDim = dim3((unsigned)p.threads);
    cfg.dynamicSmemBytes = (size_t)p.smem_bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n_split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = n_split > 1 ? attr : nullptr;
    cfg.numAttrs = n_split > 1 ? 1 : 0;
    auto go = [&](auto kern) {
        return cudaLaunchKernelEx(
            &cfg, kern, (const uint4*)q, (const uint8_t*)c.k_codes, (const uint8_t*)c.k_scales,
            (const uint8_t*)c.v_codes, (const uint8_t*)c.v_scales, q_seq, q_pos, sel_idx, sel_cnt, c.page_table,
            (int)c.page_tokens, c.page_table ? d.kv_capacity / c.page_tokens : (int64_t)0, c.n_pages, (int)d.batch,
            (int)d.n_q_heads, (int)d.n_kv_heads, d.kv_capacity, bs_log2, (int)d.top_k, group_q,
            scale * 1.4426950408889634f, items, n_split, area, (__nv_bfloat16*)out, status);
    };
    if (nt == 1)
        return tier == 0   ? go(k_sparse_attn_kv4<1, 16, 2>)
               : tier == 1 ? go(k_sparse_attn_kv4<1, 8, 2>)
                           : go(k_sparse_attn_kv4<1, 4, 2>);
    if (nt == 2) return tier == 0 ? go(k_sparse_attn_kv4<2, 8, 2>) : go(k_sparse_attn_kv4<2, 4, 2>);
    return tier == 0 ? go(k_sparse_attn_kv4<4, 8, 2>) : go(k_sparse_attn_kv4<4, 4, 2>);
}

}  // namespace qsa
