// Appending K and V rows to a cache held in 4 bits (blocks of 16 values: e2m1 codes and
// one e4m3 scale).  For each 16 values x of a row of 128:
//     s = e4m3( max|x| / 6 ) kept in [2^-9, 448],   c = e2m1( x / s ),
// both rounded to nearest even; 6 is the largest e2m1 value.  A block with a value that is
// not finite gets the scale NaN and codes 0.
//
// x / s without a division per value: r = 1 / s rounded, y = x r, which is off by at most
// 2^-23 of x / s.  A code changes at borders t of 1 to 3 significant bits.  x has 8
// significant bits and t s at most 7 + 2 (4 bits of s times an odd part of t below 8), so
// x / s is either a border exactly or at least 2^-9 of it away.  y with its mantissa
// rounded to 11 bits is therefore on the side of the border that x / s is on, and is the
// border where x / s is: the conversion then breaks the tie to even as for the quotient.
//
// Bytes only: 256 read and 72 written per row.  One thread per block of 16 (two 16-byte
// loads, one 8-byte store of codes, 8 threads fill a row's 8 scale bytes), rows in the
// order of the packed input, so reads are contiguous.  8,192 tokens of 8 KV heads (33.6 MB
// read, 9.4 written: 6.5 us at the copy rate): 13.4 us with cold caches; with a division per value
// it was 17.5.  What is left is the short CTAs' waves, a search for the sequence per row, and
// scales written 8 bytes at a time.

#include "qsa_internal.cuh"

namespace qsa {

namespace {

constexpr int kAppendThreads = 256;

// codes of 8 values in byte order, low half first
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* x)
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}\n"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}

}  // namespace

__global__ void __launch_bounds__(kAppendThreads)
k_kv4_append(const __nv_bfloat16* __restrict__ k, int64_t k_ld, const __nv_bfloat16* __restrict__ v, int64_t v_ld,
             const int32_t* __restrict__ cu_len, const int32_t* __restrict__ len_before, int batch, int n_tok,
             int n_kv_heads, int64_t kv_capacity, uint8_t* __restrict__ k_codes, uint8_t* __restrict__ k_scales,
             uint8_t* __restrict__ v_codes, uint8_t* __restrict__ v_scales, const int32_t* __restrict__ page_table,
             int page_tokens, int64_t table_ld, int64_t n_pages, unsigned* status)
{
    const int lane = threadIdx.x & 31;
    // malformed lengths are skipped below; the first CTA reports them
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < batch; s += kAppendThreads) {
            const int a = __ldg(cu_len + s), b = __ldg(cu_len + s + 1), at = __ldg(len_before + s);
            if (a < 0 || a > b || b > n_tok || at < 0 || (int64_t)at + (b - a) > kv_capacity)
                set_status(status, QSA_DEV_BAD_LEN);
        }
    // row = (token, K or V, head); a warp holds four of them
    const uint32_t row = blockIdx.x * (kAppendThreads / 8) + (threadIdx.x >> 3);
    const int blk = threadIdx.x & 7;
    const uint32_t per_tok = 2 * n_kv_heads, tok32 = row / per_tok;
    const int in_tok = (int)(row - tok32 * per_tok);
    const int tok = tok32 < (uint32_t)n_tok ? (int)tok32 : -1;
    const bool is_v = in_tok >= n_kv_heads;
    const int head = is_v ? in_tok - n_kv_heads : in_tok;
    // the values are on their way while the token's sequence is looked up
    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
    if (tok >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>((is_v ? v + tok * v_ld : k + tok * k_ld) + head * kHeadDim) + 2 * blk;
        x0 = __ldg(src);
        x1 = __ldg(src + 1);
    }
    int seq = -1, found = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int t = __shfl_sync(0xffffffffu, tok, 8 * u);
        if (t < 0) break;
        if (t != found) {
            const int s = find_sequence(batch, lane, [&](int i) { return __ldg(cu_len + i) <= t; });
            if (tok == t) seq = s;
            found = t;
        }
    }
    if (tok < 0 || seq < 0) return;
    const int a = __ldg(cu_len + seq), b = __ldg(cu_len + seq + 1), at = __ldg(len_before + seq);
    // a token of no sequence, or of one whose lengths are malformed
    if (a < 0 || tok < a || tok >= b || b > n_tok || at < 0 || (int64_t)at + (b - a) > kv_capacity) return;
    const int pos = at + (tok - a);
    int64_t dst;
    if (page_table) {
        const int page = __ldg(page_table + (int64_t)seq * table_ld + pos / page_tokens);
        if (page < 0 || page >= n_pages) {
            if (blk == 0) set_status(status, QSA_DEV_BAD_PAGE);
            return;
        }
        dst = ((int64_t)page * n_kv_heads + head) * page_tokens + pos % page_tokens;
    } else {
        dst = ((int64_t)seq * n_kv_heads + head) * kv_capacity + pos;
    }
    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    float x[16], top = 0.f;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[2 * e] = bf16lo(w[e]);
        x[2 * e + 1] = bf16hi(w[e]);
        finite = finite && (w[e] & 0x7F80u) != 0x7F80u && (w[e] & 0x7F800000u) != 0x7F800000u;
        top = fmaxf(top, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
    }
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(s8) : "f"(0.f), "f"(fmaxf(__fdiv_rn(top, 6.0f), 0x1p-9f)));
    uint32_t s16;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(s16) : "h"(s8));
    float s;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}\n" : "=f"(s) : "r"(s16));
    const float r = __frcp_rn(s);
#pragma unroll
    for (int e = 0; e < 16; ++e)   // (an infinite product stays infinite and saturates)
        x[e] = __uint_as_float((__float_as_uint(x[e] * r) + 0x1000u) & 0xFFFFE000u);
    uint2 codes = make_uint2(pack_e2m1x8(x), pack_e2m1x8(x + 8));
    if (!finite) {
        codes = make_uint2(0u, 0u);
        s8 = 0x7F;
    }
    *reinterpret_cast<uint2*>((is_v ? v_codes : k_codes) + dst * (kHeadDim / 2) + 8 * blk) = codes;
    (is_v ? v_scales : k_scales)[dst * (kHeadDim / 16) + blk] = (uint8_t)s8;
}

cudaError_t launch_kv4_append(const qsa_dims& d, const qsa_kv4_cache& c, const void* k, int64_t k_ld, const void* v,
                              int64_t v_ld, const int32_t* cu_len, const int32_t* len_before, int32_t n_tok,
                              unsigned* status, cudaStream_t st)
{
    const int64_t threads = (int64_t)n_tok * 2 * d.n_kv_heads * 8;
    k_kv4_append<<<(unsigned)((threads + kAppendThreads - 1) / kAppendThreads), kAppendThreads, 0, st>>>(
        (const __nv_bfloat16*)k, k_ld, (const __nv_bfloat16*)v, v_ld, cu_len, len_before, d.batch, n_tok, d.n_kv_heads,
        d.kv_capacity, (uint8_t*)c.k_codes, (uint8_t*)c.k_scales, (uint8_t*)c.v_codes, (uint8_t*)c.v_scales,
        c.page_table, c.page_tokens, c.page_table ? d.kv_capacity / c.page_tokens : 0, c.n_pages, status);
    return cudaGetLastError();
}

}  // namespace qsa
